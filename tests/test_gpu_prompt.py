"""kq8_prompt_attn: causal attention over packed fp16 / bf16 prompts against the
formula in 64 bits.

Tolerances.  Let u be a rounding of the type (bf16 2^-8, fp16 2^-11: finfo.eps / 2).
Products of two such numbers are exact in fp32.  A score's sum of 128 terms, its scale
and the difference to the maximum take fewer than 160 fp32 roundings (inside a matrix
instruction up to 2^-23 each) of at most A = max sum_d |q_d k_d| * scale: a weight is
off by at most 160 * 2^-23 * A of itself, by its exponential 2^-22, and by u from its
rounding.  The sums over blocks add fewer than 2 * 64 fp32 roundings.  An output is a
mean of values below max|v| with those weights: (u + 2 * 160 * 2^-23 * A + 2^-15) *
max|v| bounds its error before its own rounding, which is u of itself."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from query_decode_attention_gb300 import kq8  # noqa: E402

DEV = "cuda:0"
SCALE = 1.0 / np.sqrt(128.0)


def _inputs(total, nq, nkv, dtype, layout, seed, spread=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def fill(*shape):
        return (torch.randn(shape, generator=g, device=DEV) * spread).to(dtype)
    if layout == "fused":
        qkv = fill(total, nq + 2 * nkv, 128)
        return qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    if layout == "heads":
        return tuple(fill(h, total, 128).transpose(0, 1) for h in (nq, nkv, nkv))
    return fill(total, nq, 128), fill(total, nkv, 128), fill(total, nkv, 128)


def _reference(q, k, v, cu):
    """(float64 outputs, tolerance before the output's own rounding) per row."""
    nq, G = q.shape[1], q.shape[1] // k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    tol = torch.zeros((q.shape[0], nq, 1), dtype=torch.float64, device=DEV)
    for a, e in zip(cu, cu[1:]):
        for h in range(nq):
            qd, kd, vd = q[a:e, h].double(), k[a:e, h // G].double(), v[a:e, h // G].double()
            s = (qd @ kd.T) * SCALE
            n = e - a
            s.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=DEV).triu(1), -np.inf)
            out[a:e, h] = torch.softmax(s, -1) @ vd
            if n:
                A = float((qd.abs() @ kd.abs().T).max()) * SCALE
                tol[a:e, h] = (u + 320 * 2.0 ** -23 * A + 2.0 ** -15) * vd.abs().max()
    return out, tol


def _run(q, k, v, cu, max_len, status=None, stream=None):
    out = torch.full((q.shape[0], q.shape[1], 128), 77.0, dtype=q.dtype, device=DEV)
    kq8.kq8_prompt_attn(out, q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), max_len,
                        SCALE, status, stream)
    return out


def _check(out, q, k, v, cu):
    ref, tol = _reference(q, k, v, cu)
    got = out.double()
    n = cu[-1]
    assert bool(torch.isfinite(got[:n]).all())
    over = (got - ref).abs() - (tol + torch.finfo(q.dtype).eps / 2 * ref.abs())
    over = over[cu[0]:n]
    assert over.numel() == 0 or float(over.max()) <= 0, f"worst excess {float(over.max()):.3e}"
    assert bool((out[n:] == 77).all()) and bool((out[:cu[0]] == 77).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nkv,lens,layout", [
    (1, 1, [1], "packed"),
    (2, 2, [128], "packed"),                                 # G = 1: one tile, one block
    (1, 1, [129], "fused"),                                  # a second tile of one row
    (8, 8, [257, 1, 0, 300], "fused"),                       # G = 1, ragged, an empty sequence
    (16, 8, [506], "fused"),                                 # G = 2
    (32, 8, [1000, 77, 128, 31, 640], "fused"),              # G = 4, packed
    (6, 2, [500, 43, 42, 84, 85], "heads"),                  # G = 3: 42 tokens a tile
    (5, 1, [333, 25, 26, 50, 51], "packed"),                 # G = 5
    (12, 2, [200, 21, 42], "fused"),                         # G = 6
    (7, 1, [150, 18, 19], "heads"),                          # G = 7
    (8, 1, [700, 16, 17, 32, 33], "fused"),                  # G = 8
    (4, 2, [2050], "fused"),                                 # the ring turns over
])
def test_prompt_matches_the_formula(dtype, nq, nkv, lens, layout):
    cu = [0] + np.cumsum(lens).tolist()
    q, k, v = _inputs(cu[-1], nq, nkv, dtype, layout, seed=cu[-1] + nq)
    out = _run(q, k, v, cu, max(lens))
    _check(out, q, k, v, cu)


def test_peaked_scores_rescale_often():
    # scores of up to a hundred and growing along the prompt
    q, k, v = _inputs(900, 4, 2, torch.bfloat16, "packed", 3)
    q *= 4
    k *= torch.linspace(0.1, 4, 900, device=DEV)[:, None, None].to(k.dtype)
    _check(_run(q, k, v, [0, 900], 900), q, k, v, [0, 900])


def test_rows_outside_every_sequence_are_not_looked_at():
    cu = [5, 45, 200]
    q, k, v = _inputs(260, 8, 2, torch.bfloat16, "fused", 4)
    for t in (q, k, v):
        t[:5] = float("nan")
        t[200:] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = _run(q, k, v, cu, 155, status)
    assert kq8.kq8_read_status(status) == 0
    _check(out, q, k, v, cu)


def test_a_sequence_of_nans_stays_by_itself():
    lens = [70, 90, 130]
    cu = [0] + np.cumsum(lens).tolist()
    q, k, v = _inputs(cu[-1], 4, 2, torch.float16, "packed", 5)
    ref, tol = _reference(q, k, v, cu)
    for t in (q, k, v):
        t[70:160] = float("nan")
    got = _run(q, k, v, cu, 130).double()
    assert bool(torch.isnan(got[70:160]).all())
    for a, e in ((0, 70), (160, 290)):
        assert bool(((got - ref).abs() <= tol + torch.finfo(q.dtype).eps / 2 * ref.abs())[a:e].all())


def test_keys_behind_a_row_may_be_anything():
    q, k, v = _inputs(300, 2, 1, torch.bfloat16, "packed", 6)
    ref, tol = _reference(q, k, v, [0, 300])
    k[250:] = float("nan")
    got = _run(q, k, v, [0, 300], 300).double()
    assert bool(((got - ref).abs() <= tol + 2.0 ** -8 * ref.abs())[:250].all())


def test_loose_bound_and_empty_calls():
    q, k, v = _inputs(64, 4, 4, torch.bfloat16, "packed", 7)
    _check(_run(q, k, v, [0, 30, 64], 10 ** 6), q, k, v, [0, 30, 64])
    assert bool((_run(q, k, v, [0], 64) == 77).all())
    assert bool((_run(q, k, v, [0, 0, 0], 64) == 77).all())
    assert bool((_run(q, k, v, [0, 64], 0) == 77).all())


@pytest.mark.parametrize("cu", [[0, 40, 30], [0, 40, 65], [0, 40, 200], [0, 40, 2 ** 31 - 1]])
def test_bad_offsets_are_reported_and_skipped(cu):
    q, k, v = _inputs(64, 4, 2, torch.bfloat16, "packed", 8)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = _run(q, k, v, cu, 64, status)
    assert kq8.kq8_read_status(status) == kq8.KQ8_STATUS_BAD_SEQLEN
    assert bool((out[40:] == 77).all())
    ref, tol = _reference(q[:40], k[:40], v[:40], [0, 40])
    assert bool(((out[:40].double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())
    # too long for the bound
    out = _run(q, k, v, [0, 40, 64], 39, status)
    assert kq8.kq8_read_status(status) == kq8.KQ8_STATUS_BAD_SEQLEN
    assert bool((out[:40] == 77).all()) and bool((out[40:] != 77).any())


def test_streams_and_graph():
    cu = [0, 300, 420]
    q, k, v = _inputs(420, 8, 2, torch.bfloat16, "fused", 9)
    want = _run(q, k, v, cu, 300)
    _check(want, q, k, v, cu)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in range(2)]
    torch.cuda.synchronize()
    for st, o in zip(s, outs):
        for _ in range(4):
            kq8.kq8_prompt_attn(o, q, k, v, cut, 300, SCALE, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    with torch.cuda.stream(s[0]):
        g = torch.cuda.CUDAGraph()
        outs[0].zero_()
        with torch.cuda.graph(g, stream=s[0]):
            kq8.kq8_prompt_attn(outs[0], q, k, v, cut, 300, SCALE)
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    r = np.random.default_rng(2000 + seed)
    for _ in range(6):
        nkv, G = int(r.choice([1, 2, 3])), int(r.integers(1, 9))
        lens = [int(2 ** r.uniform(-1, 10.5)) for _ in range(int(r.integers(1, 7)))]
        lens[0] = max(lens[0], 1)
        first, behind = int(r.integers(4)), int(r.integers(4))
        cu = (first + np.concatenate([[0], np.cumsum(lens)])).tolist()
        q, k, v = _inputs(cu[-1] + behind, G * nkv, nkv, [torch.bfloat16, torch.float16][seed % 2],
                          str(r.choice(["fused", "heads", "packed"])), seed=int(r.integers(1 << 20)))
        _check(_run(q, k, v, cu, max(lens) + int(r.integers(200))), q, k, v, cu)
