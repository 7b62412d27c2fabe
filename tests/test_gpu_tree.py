"""kq8_tree_attn: attention of drafted tokens over the paged q8 cache, against the
method in 64 bits (Q's codes by the method's fp32 rule, everything after them in
float64) on the very codes the cache holds.

Tolerances.  Let A be the largest sum_b |dot_b qsc_b| * ks/127 * scale of a row.  A
score takes 4 multiply-adds, 3 roundings of its token's multiplier and one product:
8 roundings of 2^-24 of at most A, so a weight e^(s - max) is off by at most 8 * 2^-24
* A of itself.  Its exponential (2^-22), its fp16 hi + lo parts (2^-22) and the sums
(in these cases fewer than 100 fp32 additions a partial sum, 2^-24 or, inside a matrix
instruction, 2^-23 each) add less than 2^-17.  An output is a mean of values below
max|v| with those weights, so numerator and denominator together give (16 * 2^-24 * A
+ 2^-16) * max|v|.

bf16 outputs have their operands rounded to fp16, u = 2^-11 of each: the weights, and with
more than 32 rows also Q and K with their scales and V with its.  With A2 the largest
sum_d |q_d k_d| * scale, a score is off by at most 2 u A2 more and a weight by 2 u A2 + u of
itself, so the output by 2 (2 u A2 + u) + u of max|v|.  That is the worst case; as the
roundings are independent the whole output is much nearer, and is held to 2^-8 in the
2-norm: its own rounding is at most 2^-8 of each value, 2^-8 / sqrt(3) in the mean, and the
operands' add u / sqrt(3) for each of the three factors and sqrt(2) u / sqrt(3) * |s| with
scores |s| of a few units: together less than 2^-8.  A 16-bit output is rounded once:
finfo.eps / 2 of itself."""
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


class Case:
    """Sequences of lens[b] cached tokens, the last nodes[b] of them drafts."""

    def __init__(self, nq, nkv, lens, nodes, dtype, kv_bs=32, seed=0, words=None, spread=1.0,
                 layout="fused", extra_rows=0):
        r = np.random.default_rng(seed)
        self.nq, self.nkv, self.lens, self.nodes = nq, nkv, list(lens), list(nodes)
        self.dtype, self.kv_bs = dtype, kv_bs
        need = [-(-n // kv_bs) for n in lens]
        pages = sum(need) + 2
        order = r.permutation(pages)
        self.table = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
        o = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[o:o + n]
            o += n
        self.slots = [self.table[b, np.arange(n) // kv_bs].astype(np.int64) * kv_bs
                      + np.arange(n) % kv_bs for b, n in enumerate(lens)]
        self.cache = kq8.PagedKVCache(pages, nkv, kv_bs, DEV)
        # every row no token owns holds the worst: extreme codes, NaN and inf maxima
        self.cache.k.fill_(-127)
        self.cache.v.fill_(127)
        self.cache.kscale.fill_(float("nan"))
        self.cache.vscale.fill_(float("inf"))
        T = sum(lens)
        if T:
            kv = torch.tensor(r.standard_normal((2, T, nkv, 128)) * spread, dtype=torch.float32,
                              device=DEV)
            kq8.kq8_write_kv(self.cache, kv[0], kv[1], _ints(np.concatenate(self.slots)))
        self.total = sum(nodes)
        self.off = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.words = words if words else max(1, -(-max(nodes, default=1) // 32))
        bits = r.random((self.total, self.words * 32)) < 0.5
        for b in range(len(lens)):
            for i in range(nodes[b]):
                bits[self.off[b] + i, i] = True
        self.bits = bits
        rows = self.total + extra_rows
        if layout == "fused":
            q = torch.empty((rows, nq + 3, 128), dtype=dtype, device=DEV)[:, 1:nq + 1]
        elif layout == "heads":
            q = torch.empty((nq, rows, 128), dtype=dtype, device=DEV).transpose(0, 1)
        else:
            q = torch.empty((rows, nq, 128), dtype=dtype, device=DEV)
        q.copy_(torch.tensor(r.standard_normal((rows, nq, 128)) * 1.5))
        self.q = q
        self.out = torch.full((rows, nq, 128), 77.0, dtype=dtype, device=DEV)

    def mask(self, rows=None):
        b = np.pad(self.bits, ((0, (rows or self.total) - self.total), (0, 0)))
        w = (b.reshape(b.shape[0], self.words, 32).astype(np.uint64)
             << np.arange(32, dtype=np.uint64)).sum(-1)
        return torch.tensor(w.astype(np.uint32).view(np.int32), device=DEV)

    def run(self, mask=True, max_len=None, max_nodes=None, ws=None, stream=None, **kw):
        max_len = max(self.lens, default=0) if max_len is None else max_len
        max_nodes = max(self.nodes, default=0) if max_nodes is None else max_nodes
        table, lens, off = _ints(self.table), _ints(self.lens), _ints(self.off)
        table = kw.get("table", table)
        lens = kw.get("lens", lens)
        off = kw.get("off", off)
        if ws is None:
            ws = kq8.new_workspace(kq8.kq8_tree_workspace_bytes(len(self.lens), self.nq, self.nkv,
                                                                max_len, max_nodes), DEV)
        kq8.kq8_tree_attn(self.out, self.q, self.cache, table, lens, off,
                          self.mask(self.q.shape[0]) if mask else None, max_len, max_nodes, SCALE,
                          ws, stream=stream)
        return kq8.kq8_read_status(ws)

    def reference(self, mask=True, skip_tokens=()):
        """(outputs float64 [total, nq, 128], the fp32 tolerance of each row)."""
        x = self.q[:self.total].float().cpu().numpy().reshape(self.total, self.nq, 4, 32)
        m = np.abs(x).max(-1, keepdims=True)
        m = np.where(m < np.float32(1e-6), np.float32(1), m)
        code = np.trunc(np.clip(x * (np.float32(127) / m), np.float32(-128), np.float32(127)))
        qd = code.astype(np.float64) * (m * (np.float32(1) / np.float32(127))).astype(np.float64)
        qd = qd.reshape(self.total, self.nq, 128)
        G = self.nq // self.nkv
        out = np.zeros((self.total, self.nq, 128))
        tol, self.more = np.zeros((self.total, 1, 1)), np.zeros((self.total, 1, 1))
        for b, n in enumerate(self.lens):
            nb, o = self.nodes[b], self.off[b]
            if nb == 0:
                continue
            k8, ks, v8, vs = paged.unpack(self.cache, self.slots[b])
            k = k8.astype(np.float64) * (ks.astype(np.float64) / 127)[..., None]
            v = v8.astype(np.float64) * (vs.astype(np.float64) / 127)[..., None]
            see = np.ones((nb, n), bool)
            if mask:
                see[:, n - nb:] = self.bits[o:o + nb, :nb]
            else:
                see[:, n - nb:] = np.tril(np.ones((nb, nb), bool))
            for t in skip_tokens:
                see[:, t] = False
            a2 = np.einsum("ihd,thd->iht", np.abs(qd[o:o + nb]), np.abs(np.repeat(k, G, 1))).max()
            if self.dtype == torch.bfloat16:
                u = 2.0 ** -11
                self.more[o:o + nb] = (2 * (2 * u * a2 * SCALE + u) + u) * np.abs(v).max()
            a = sum(np.abs(np.einsum("ihd,thd->iht", qd[o:o + nb, :, e:e + 32],
                                     np.repeat(k, G, 1)[..., e:e + 32])) for e in range(0, 128, 32))
            tol[o:o + nb] = (2.0 ** -20 * a.max() * SCALE + 2.0 ** -16) * np.abs(v).max()
            s = np.einsum("ihd,thd->iht", qd[o:o + nb], np.repeat(k, G, 1)) * SCALE
            s = np.where(see[:, None], s, -np.inf)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - np.where(np.isinf(top), 0.0, top))
            den = p.sum(-1, keepdims=True)
            p = p / np.where(den == 0, 1.0, den)
            out[o:o + nb] = np.einsum("iht,thd->ihd", p, np.repeat(v, G, 1))
        return out, tol

    def check(self, ref, tol):
        got = self.out[:self.total].double().cpu().numpy()
        if self.dtype != torch.float32:
            tol = tol + self.more
            tol = tol + torch.finfo(self.dtype).eps / 2 * np.abs(ref)
        assert np.all(np.isfinite(got))
        if self.dtype == torch.bfloat16:
            assert np.linalg.norm(got - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
        err = np.abs(got - ref) - tol
        assert np.all(err <= 0), f"worst excess {err.max():.3e}"
        # rows behind the last sequence stay as they were
        assert bool((self.out[self.total:] == 77).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nkv,lens,nodes,kv_bs", [
    (2, 2, [1], [1], 32),                                # one token, itself
    (16, 8, [300, 77, 1000], [8, 5, 13], 32),            # G = 2
    (32, 8, [2000, 64, 33], [26, 64, 1], 64),            # G = 4, a sequence that is all drafts
    (8, 1, [500, 40, 31], [3, 40, 31], 32),              # G = 8, all drafts
    (6, 2, [200, 999], [100, 7], 128),                   # G = 3, several mask words
    (5, 1, [333], [33], 256),                            # G = 5
    (4, 4, [31, 32, 33, 63, 64, 65], [1, 2, 31, 32, 33, 65], 32),  # sub-tile borders, G = 1
    (7, 1, [130], [1], 32),                              # G = 7, one node
    (4, 1, [900, 5000], [12, 4], 32),                    # 48 rows; a sequence in several chunks
    (8, 2, [3000, 129, 127], [8, 8, 5], 64),             # 32 rows, several chunks
    (24, 3, [4097, 300], [16, 2], 32),                   # 128 rows, G = 8
])
def test_tree_matches_the_method(dtype, nq, nkv, lens, nodes, kv_bs):
    c = Case(nq, nkv, lens, nodes, dtype, kv_bs, seed=sum(lens) + nq)
    assert c.run() == 0
    c.check(*c.reference())


@pytest.mark.parametrize("layout", ["fused", "heads", "packed"])
def test_strides_extra_rows_and_loose_bounds(layout):
    c = Case(8, 2, [400, 90], [9, 17], torch.bfloat16, seed=5, layout=layout, extra_rows=3, words=3)
    assert c.run(max_len=416, max_nodes=70) == 0
    c.check(*c.reference())


def test_chain_without_a_mask():
    c = Case(16, 8, [700, 45], [40, 45], torch.float32, seed=6)
    assert c.run(mask=False) == 0
    c.check(*c.reference(mask=False))


@pytest.mark.parametrize("nkv", [2, 4])
def test_rows_that_see_nothing_give_zero(nkv):
    # a sequence that is all drafts (no committed token), some nodes with an empty mask
    c = Case(4, nkv, [20, 50], [20, 6], torch.bfloat16, seed=7)
    c.bits[[0, 3, 19]] = False
    c.bits[[21]] = False       # sees its committed tokens only
    assert c.run() == 0
    ref, tol = c.reference()
    assert np.all(ref[[0, 3, 19]] == 0)
    assert bool((c.out[[0, 3, 19]] == 0).all())
    c.check(ref, tol)


@pytest.mark.parametrize("nodes", [5, 12, 40])
def test_masked_draft_rows_may_hold_anything(nodes):
    # node 2's K and V rows hold inf and NaN; nodes that do not see it are untouched by them
    c = Case(4, 2, [60], [nodes], torch.float32, seed=8)
    c.bits[:, 2] = False
    ref, tol = c.reference()
    slot = int(c.slots[0][60 - nodes + 2])
    c.cache.kscale[slot // 32, :, slot % 32] = float("nan")
    c.cache.vscale[slot // 32, :, slot % 32] = float("inf")
    assert c.run() == 0
    c.check(ref, tol)


def test_bits_past_the_last_node_are_ignored():
    c = Case(4, 2, [90, 70], [5, 33], torch.float32, seed=9, words=2)
    c.bits[:, :] |= np.arange(64) >= 33
    c.bits[:5, 5:] = True
    assert c.run() == 0
    c.check(*c.reference())


def test_one_node_equals_the_decode():
    c = Case(16, 8, [900, 5, 64], [1, 1, 1], torch.float32, seed=10, layout="packed")
    assert c.run() == 0
    ws = kq8.new_workspace(kq8.kq8_decode_workspace_bytes(3, 16, 8, 900), DEV)
    dec = torch.empty_like(c.out)
    kq8.kq8_decode_attn(dec, c.q, c.cache, _ints(c.table), _ints(c.lens), 900, SCALE, ws)
    tol = c.reference()[1].max()
    assert float((dec - c.out).abs().max()) <= 2 * tol  # both are fp32 forms of one sum


@pytest.mark.parametrize("nodes", [4, 8, 20])  # 16, 32, 80 rows: both kernels
def test_large_scores_and_v_steps(nodes):
    # keys and values over many octaves: the running maximum jumps, the V steps' exponent grows
    c = Case(8, 2, [3000], [nodes], torch.float32, seed=11)
    f = torch.tensor(2.0) ** torch.randint(-20, 3, c.cache.vscale.shape)
    c.cache.vscale.mul_(f.to(DEV))
    c.cache.kscale.mul_((torch.tensor(2.0) ** torch.randint(-4, 4, c.cache.kscale.shape)).to(DEV))
    assert c.run() == 0
    c.check(*c.reference())


@pytest.mark.parametrize("nodes", [3, 8, 11, 30, 60])  # 12, 32, 44, 120, 240 rows
def test_long_context_many_chunks(nodes):
    c = Case(4, 1, [20011], [nodes], torch.bfloat16, seed=12)
    assert c.run() == 0
    c.check(*c.reference())
    first = c.out.clone()
    for _ in range(3):  # tickets and partials reused
        c.out.zero_()
        assert c.run() == 0
        assert torch.equal(first, c.out)


def test_zero_nodes_and_empty_batch():
    c = Case(4, 2, [100, 50, 0], [4, 0, 0], torch.float32, seed=13)
    assert c.run() == 0
    c.check(*c.reference())
    e = Case(4, 2, [], [], torch.float32, seed=14)
    assert e.run() == 0


@pytest.mark.parametrize("lens,off", [
    ([100, 3], [0, 4, 9]),       # more drafts than tokens
    ([100, -1], [0, 4, 9]),
    ([100, 201], [0, 4, 9]),     # past max_seq_len
    ([100, 50], [0, 4, 40]),     # past total_q
    ([100, 50], [0, 4, 2]),      # offsets descend
])
@pytest.mark.parametrize("nq", [2, 16])
def test_bad_sequence_is_reported_and_skipped(lens, off, nq):
    c = Case(nq, 2, [100, 50], [4, 5], torch.float32, seed=15)
    ref, tol = c.reference()
    table = np.full((2, 7), -1, np.int32)
    table[:, :c.table.shape[1]] = c.table
    st = c.run(lens=_ints(lens), off=_ints(off), table=_ints(table), max_len=200, max_nodes=9)
    assert st == kq8.KQ8_STATUS_BAD_SEQLEN
    assert bool((c.out[4:] == 77).all())
    got = c.out[:4].double().cpu().numpy()
    assert np.all(np.abs(got - ref[:4]) <= tol[:4])


@pytest.mark.parametrize("bad", [-1, 10 ** 9, "pages"])
@pytest.mark.parametrize("nq", [4, 16])
def test_bad_page_is_left_out(bad, nq):
    c = Case(nq, 2, [200, 70], [4, 5], torch.float32, seed=16)
    ref, tol = c.reference()
    table = c.table.copy()
    table[0, 1] = c.cache.num_pages if bad == "pages" else bad
    assert c.run(table=_ints(table)) == kq8.KQ8_STATUS_BAD_PAGE
    got = c.out.double().cpu().numpy()
    assert np.all(np.abs(got[4:] - ref[4:]) <= tol[4:])  # the other sequence is whole
    # tokens 32 .. 63 of sequence 0 are left out
    c.nodes = [4, 0]
    part, tol = c.reference(skip_tokens=range(32, 64))
    assert np.all(np.abs(got[:4] - part[:4]) <= tol[:4])


def test_two_streams_with_their_own_workspaces_and_a_graph():
    a = Case(8, 2, [5000, 700], [12, 7], torch.bfloat16, seed=17)
    b = Case(8, 2, [3333], [30], torch.float16, seed=18)
    for c in (a, b):
        assert c.run() == 0
    want = [a.out.clone(), b.out.clone()]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = []
    for c in (a, b):
        ws = kq8.new_workspace(kq8.kq8_tree_workspace_bytes(len(c.lens), 8, 2, max(c.lens),
                                                            max(c.nodes)), DEV)
        args.append((c, _ints(c.table), _ints(c.lens), _ints(c.off), c.mask(), ws))
    torch.cuda.synchronize()

    def call(c, table, lens, off, mask, ws):
        kq8.kq8_tree_attn(c.out, c.q, c.cache, table, lens, off, mask, max(c.lens), max(c.nodes),
                          SCALE, ws)
    for _ in range(5):  # overlapping calls
        for st, ar in zip(s, args):
            ar[0].out.zero_()
    torch.cuda.synchronize()
    for st, ar in zip(s, args):
        with torch.cuda.stream(st):
            for _ in range(5):
                call(*ar)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    # one workspace in two graphs of one stream, replayed in turn
    big = max((ar[-1] for ar in args), key=lambda w: w.numel())
    graphs = []
    with torch.cuda.stream(s[0]):
        for ar in args:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s[0]):
                call(*ar[:-1], big)
            graphs.append(g)
        for _ in range(3):
            a.out.zero_(), b.out.zero_()
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_sums_that_leave_the_accumulator():
    """Shares of 40 steps of 128 tokens: hi and lo parts take O out of the accumulator twice
    on the way; a third of the tokens raises the reference late."""
    nkv, B = 8, 2
    n = torch.cuda.get_device_properties(0).multi_processor_count * 40 * 128 // (nkv * B) + 77
    c = Case(16, nkv, [n, n - 500], [20, 18], torch.float32, seed=37)
    late = torch.tensor(np.concatenate([s[2 * len(s) // 3:] for s in c.slots]), device=DEV)
    k, v = (torch.empty((len(late), nkv, 128), device=DEV) for _ in range(2))
    kq8.kq8_read_kv(c.cache, k, v, late.int())
    kq8.kq8_write_kv(c.cache, 2 * k, v, late.int())
    assert c.run() == 0
    # the method in float64 on the GPU, one head at a time
    ks, vs = (torch.empty((sum(c.lens), nkv, 128), device=DEV) for _ in range(2))
    kq8.kq8_read_kv(c.cache, ks, vs, _ints(np.concatenate(c.slots)))
    x = c.q.reshape(c.total, 16, 4, 32)
    m = x.abs().amax(-1, keepdim=True)
    code = torch.trunc((x * (torch.tensor(127.0, device=DEV) / m)).clamp(-128, 127)).double()
    qd = (code * (m * (torch.tensor(1.0, device=DEV) / 127)).double()).reshape(c.total, 16, 128)
    ref, at = torch.empty_like(qd), 0
    for b, n in enumerate(c.lens):
        nb, o = c.nodes[b], int(c.off[b])
        see = torch.tensor(c.bits[o:o + nb, :nb], device=DEV)
        for h in range(16):
            kd, vd = ks[at:at + n, h // 2].double(), vs[at:at + n, h // 2].double()
            s = qd[o:o + nb, h] @ kd.T * SCALE
            s[:, n - nb:][~see] = -torch.inf
            ref[o:o + nb, h] = torch.softmax(s, -1) @ vd
        at += n
    # a chain of 16 steps is 256 additions of half a last place, cut off: 256 * 2^-24 of the
    # sums' size, which the later chains' own sums (rounded to nearest) hardly add to; the
    # read rows are one rounding, 2^-24, off, scores with it
    assert float((c.out.double() - ref).norm()) <= 2.0 ** -16 * float(ref.norm())


def test_all_forms_share_a_workspace_and_replay():
    """One and two 16-row tiles a warp, one and two 128-row tiles, hi and lo parts: each
    captured, then replayed in turn over one workspace, with other queries at the second
    time."""
    cases = [Case(4, 2, [3000, 100], [5, 3], torch.float32, seed=31),
             Case(8, 2, [2500], [7], torch.bfloat16, seed=32),
             Case(8, 2, [4000, 77, 900], [20, 9, 32], torch.bfloat16, seed=33),
             Case(16, 2, [1500, 2100], [31, 17], torch.bfloat16, seed=34),
             Case(8, 2, [2222, 640], [40, 11], torch.float32, seed=35)]
    size = max(kq8.kq8_tree_workspace_bytes(len(c.lens), c.nq, 2, max(c.lens), max(c.nodes))
               for c in cases)
    ws = kq8.new_workspace(size, DEV)
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for c in cases:
            args = (_ints(c.table), _ints(c.lens), _ints(c.off), c.mask(), max(c.lens), max(c.nodes))
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                kq8.kq8_tree_attn(c.out, c.q, c.cache, *args, SCALE, ws)
            graphs.append((g, args))
        for turn in range(2):
            for c, (g, _) in zip(cases, graphs):
                g.replay()
            assert kq8.kq8_read_status(ws) == 0
            for c in cases:
                c.check(*c.reference())
                c.q.copy_(c.q.flip(0))
    torch.cuda.synchronize()


def test_out_over_q_is_refused():
    c = Case(8, 2, [100], [4], torch.bfloat16, layout="packed", seed=36)
    c.out = c.q
    with pytest.raises(kq8.Kq8Error):
        c.run()


@pytest.mark.parametrize("nodes,dtype", [(4, torch.bfloat16), (20, torch.bfloat16), (20, torch.float32)])
def test_pages_past_2_gib(nodes, dtype):
    """The same tokens in the first pages of a pool and in its last ones, past 2^31 bytes of
    K and of V: the same outputs bit for bit."""
    nq, nkv, kv_bs, n = 32, 8, 256, 600
    pages = (1 << 31) // (kv_bs * nkv * 128) + 8
    cache = kq8.PagedKVCache(pages, nkv, kv_bs, DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    k, v = (torch.randn((n, nkv, 128), generator=g, device=DEV) for _ in range(2))
    q = torch.randn((nodes, nq, 128), generator=g, device=DEV).to(dtype)
    outs = []
    for first in (0, pages - 3):
        at = torch.arange(n, dtype=torch.int32, device=DEV)
        kq8.kq8_write_kv(cache, k, v, at + first * kv_bs)
        out = torch.zeros_like(q)
        ws = kq8.new_workspace(kq8.kq8_tree_workspace_bytes(1, nq, nkv, n, nodes), DEV)
        kq8.kq8_tree_attn(out, q, cache, _ints([[first, first + 1, first + 2]]), _ints([n]),
                          _ints([0, nodes]), None, n, nodes, SCALE, ws)
        assert kq8.kq8_read_status(ws) == 0
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and bool((outs[0] != 0).any())


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(seed):
    r = np.random.default_rng(1000 + seed)
    for _ in range(4):
        nkv, G, B = int(r.choice([1, 2, 3, 8])), int(r.integers(1, 9)), int(r.integers(1, 6))
        lens = [int(2 ** r.uniform(0, 11)) for _ in range(B)]
        most = int(r.choice([3, 9, 33, 70, 200]))
        nodes = [int(r.integers(0, min(n, most) + 1)) for n in lens]
        nodes[0] = max(nodes[0], 1)
        c = Case(G * nkv, nkv, lens, nodes, [torch.float32, torch.bfloat16, torch.float16][seed % 3],
                 kv_bs=int(r.choice([32, 64, 128, 256])), seed=int(r.integers(1 << 20)),
                 layout=str(r.choice(["fused", "heads", "packed"])), extra_rows=int(r.integers(3)))
        mask = bool(r.random() < 0.75)
        assert c.run(mask=mask) == 0
        c.check(*c.reference(mask=mask))
