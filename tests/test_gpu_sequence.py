"""Sequence operators on the GPU against their plain 64-bit forms
(sequence_ref.py, where the tolerances are derived): dense embedding lookup and
gradient, layer norm, attention over the keys of each bag, and the attention
pooling of a table's bags built from them."""
import math
import threading
import time

import pytest
import torch

import sequence_ref as S

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def R():
    import recommender_sparse_embedding_b200 as R
    from recommender_sparse_embedding_b200 import build
    build.build()
    assert torch.cuda.is_available()
    R.load()
    R.sequence_status_sync()
    return R


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, dtype, g, mul=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * mul).to(dtype)


# ------------------------------------------------------------------ dense embedding
@pytest.mark.parametrize("wt,ot", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("N,V,D", [(0, 5, 8), (1, 1, 1), (3, 7, 33), (64, 1000, 1024), (4097, 300, 40),
                                   (100000, 5000, 64), (30, 11, 2056)])
def test_embed_lookup(R, wt, ot, N, V, D):
    g = _gen(N + D)
    w = _randn((V, D), wt, g)
    t = torch.randint(-1, V, (N,), device="cuda", generator=g)
    scale = 0.375 if N % 2 else math.sqrt(D)
    out = R.embed_lookup(w, t, scale=scale, out_dtype=ot)
    R.sequence_status_sync()
    want = S.lookup(w, t, scale, -1)
    # the factor and the product round to fp32, the result to its type
    S.close(out, want, (S.half_step(ot) * 1.001 + 2 * S.F32) * want.abs() + (2.0 ** -24 if ot == F16 else 0), "lookup")


def test_embed_lookup_padding_and_bad_tokens(R):
    g = _gen(3)
    w = _randn((10, 24), F32, g)
    w[4] = math.nan
    t = torch.tensor([[4, 0], [9, 4]], device="cuda")
    out = R.embed_lookup(w, t, padding=4)  # a padding token reads zeros, whatever its row holds
    R.sequence_status_sync()
    assert torch.equal(out[0, 0], torch.zeros(24, device="cuda")) and torch.equal(out[1, 0], w[9])
    out = R.embed_lookup(w, torch.tensor([10, 1, -7, 2**40], device="cuda"))
    with pytest.raises(R.RecisError):
        R.sequence_status_sync()
    R.sequence_status_sync()  # cleared
    assert torch.equal(out[1], w[1]) and not out[[0, 2, 3]].any()


def test_embed_lookup_into_strided_rows_and_misaligned_weight(R):
    g = _gen(4)
    wide = torch.zeros((50, 96), device="cuda", dtype=BF16)
    w = _randn((20 * 16 + 1,), BF16, g)[1:].view(20, 16)  # rows off the 16-byte boundary
    t = torch.randint(0, 20, (50,), device="cuda", generator=g)
    R.embed_lookup(w, t, out=wide[:, 40:56])
    assert torch.equal(wide[:, 40:56], w[t])
    assert not wide[:, :40].any() and not wide[:, 56:].any()


def _tokens(kind, N, V, g):
    if kind == "one":
        return torch.full((N,), V - 1, device="cuda")
    if kind == "padding":
        return torch.full((N,), -1, device="cuda")
    if kind == "hot":  # half the positions hold one token, the rest spread, some padding
        t = torch.randint(-1, V, (N,), device="cuda", generator=g)
        return torch.where(torch.rand(N, device="cuda", generator=g) < 0.5, V // 2, t)
    return torch.randint(0, V, (N,), device="cuda", generator=g)


@pytest.mark.parametrize("gt,ot", [(F32, F32), (BF16, F32), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("kind,N,V,D", [
    ("even", 0, 5, 8), ("even", 1, 1, 1), ("hot", 1024, 40, 72), ("hot", 1025, 40, 72), ("one", 1000, 3, 16),
    ("one", 5000, 70000, 16), ("even", 20011, 31, 33), ("hot", 70000, 1 << 17, 64), ("padding", 3000, 9, 8),
    ("even", 4096, 1 << 21, 8), ("hot", 9999, 1000, 520), ("even", 300, 7, 300), ("hot", 700001, 3000, 8)])
def test_embed_grad(R, gt, ot, kind, N, V, D):
    g = _gen(N + V + D)
    t = _tokens(kind, N, V, g)
    grad = _randn((N, D), gt, g)
    scale = 1.5
    out = R.embed_grad(t, grad, V, scale=scale, dtype=ot)
    again = R.embed_grad(t, grad, V, scale=scale, dtype=ot)
    R.sequence_status_sync()
    assert torch.equal(out, again)  # the order of the sums does not depend on scheduling
    want, mag = S.embed_grad(t, grad, V, scale, -1)
    # at most 128 terms a thread in fp32, then fp64; the scaled sum rounds to fp32 and to the type
    S.close(out, want, 132 * S.F32 * mag + S.half_step(ot) * 1.01 * want.abs() + (2.0 ** -24 if ot == F16 else 0), "grad")


@pytest.mark.parametrize("N", [500, 6000])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_embed_grad_accumulates(R, N, dt):
    g = _gen(N)
    V, D = 3000, 48
    t = _tokens("hot", N, V, g)
    t[:5] = torch.tensor([V, -9, 2**33, -1, 0])  # three of them out of range
    grad = _randn((N, 2 * D), F32, g)[:, D:]      # rows of a wider tensor
    old = _randn((V, D), dt, g)
    out = old.clone()
    res = R.embed_grad(t, grad, V, out=out, accumulate=True)
    with pytest.raises(R.RecisError):
        R.sequence_status_sync()
    assert res is out
    want, mag = S.embed_grad(t, grad, V, 1.0, -1)
    untouched = mag.sum(1) == 0
    assert torch.equal(out[untouched], old[untouched])
    want = want + old.double()
    S.close(out, want, 132 * S.F32 * (mag + old.double().abs()) + S.half_step(dt) * 1.01 * want.abs(), "accumulated")


@pytest.mark.parametrize("N", [700, 5000])
def test_embed_grad_does_not_read_padding_rows(R, N):
    g = _gen(N + 1)
    t = _tokens("hot", N, 60, g)
    grad = _randn((N, 32), BF16, g)
    want = R.embed_grad(t, grad, 60)
    grad[t == -1] = math.nan
    assert (t == -1).any() and torch.equal(R.embed_grad(t, grad, 60), want)


# ------------------------------------------------------------------ layer norm
NORM_SIZES = [(1, 1), (5, 7), (64, 256), (1000, 8), (257, 40), (33, 128), (300, 1001), (70, 4096), (9, 8192),
              (5, 16384), (3, 5003), (4, 40000), (20000, 16), (2, 512), (40, 520), (2500, 2048), (1700, 8192),
              (3001, 300), (1300, 1000), (1250, 4096), (1210, 2600)]


@pytest.mark.parametrize("xt,yt,wt", [(F32, F32, F32), (F32, BF16, F32), (BF16, BF16, BF16), (F16, F16, F32),
                                      (BF16, F32, F16)])
@pytest.mark.parametrize("M,D", NORM_SIZES)
def test_layer_norm(R, M, D, xt, yt, wt):
    g = _gen(M * 7 + D)
    x = _randn((M, D), xt, g, 2.0) + 0.5
    x = x.to(xt)
    w, b = (_randn((D,), wt, g) + 1).to(wt), _randn((D,), wt, g)
    gy = _randn((M, D), yt, g)
    y, mean, rstd = R.layer_norm(x, w, b, eps=1e-5, out_dtype=yt)
    dx, dw, db = R.layer_norm_backward(gy, x, mean, rstd, w, b)
    ref = S.Norm(x, w, b, 1e-5)
    S.close(mean, ref.mean, ref.mean_err + S.F32 * ref.mean.abs(), "mean")
    S.close(rstd, ref.rstd, ref.rstd_err, "rstd")
    tiny = 2.0 ** -24
    S.close(y, ref.y, ref.y_err * 1.01 + S.half_step(yt) * 1.01 * ref.y.abs() + (tiny if yt == F16 else 0), "y")
    # rows a thread adds in fp32: those of one block, then fp64
    n_rows = M // 100 + 64
    (rx, ex), (rw, ew), (rb, eb) = ref.back(gy, n_rows)
    S.close(dx, rx, ex * 1.01 + S.half_step(xt) * 1.01 * rx.abs() + (tiny if xt == F16 else 1e-37), "grad_x")
    S.close(dw, rw, ew * 1.01 + S.half_step(wt) * 1.01 * rw.abs() + tiny * (wt == F16), "grad_weight")
    S.close(db, rb, eb * 1.01 + S.half_step(wt) * 1.01 * rb.abs() + tiny * (wt == F16), "grad_bias")
    again = R.layer_norm_backward(gy, x, mean, rstd, w, b)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("D", [6112, 6120, 6144])
@pytest.mark.parametrize("xt,yt", [(F16, BF16), (BF16, F16)])  # types no wider row is normalised in before
def test_layer_norm_parameters_that_just_fit_the_default_shared_memory(R, xt, yt, D):
    """Weight and bias take 48 KB of shared memory at 6144 columns, the block's
    sums some more."""
    g = _gen(D)
    x, w, b = _randn((3, D), xt, g), _randn((D,), F32, g), _randn((D,), F32, g)
    y = R.layer_norm(x, w, b, out_dtype=yt)[0]
    ref = S.Norm(x, w, b, 1e-5)
    S.close(y, ref.y, ref.y_err * 1.01 + S.half_step(yt) * 1.01 * ref.y.abs() + (2.0 ** -24 if yt == F16 else 0), "y")


def test_layer_norm_from_two_threads(R):
    """Widths whose parameters need more than 48 KB of shared memory each, from two
    host threads at once."""
    g = _gen(12)
    xs = [_randn((2, D), F32, g) for D in (6400, 8000)]
    want = [R.layer_norm(x)[0] for x in xs]
    torch.cuda.synchronize()
    L, failed = R.load(), []

    def calls(x, y):  # the entry point itself, which runs outside the interpreter's lock
        got = torch.empty_like(x)
        M, D = x.shape
        for _ in range(20000):
            if L.recis_layer_norm(x.data_ptr(), 0, D, M, D, None, None, 0, 1e-5, got.data_ptr(), 0, D, None, None,
                                  torch.cuda.current_stream().cuda_stream) != R.OK:
                failed.append(L.recis_last_error_string())
        torch.cuda.synchronize()
        if not torch.equal(got, y):
            failed.append("other values")

    threads = [threading.Thread(target=calls, args=a) for a in zip(xs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, (len(failed), failed[0])


def test_layer_norm_strided_rows_and_no_parameters(R):
    g = _gen(8)
    buf = _randn((40, 3, 48), F32, g)
    x, gy = buf[:, 1, 8:32], _randn((40, 64), BF16, g)[:, 3:27]  # gy's rows are off the 16-byte boundary
    y = torch.zeros((40, 32), dtype=BF16, device="cuda")
    _, mean, rstd = R.layer_norm(x, out=y[:, 8:])
    ref = S.Norm(x, None, None, 1e-5)
    S.close(y[:, 8:], ref.y, ref.y_err + S.half_step(BF16) * 1.01 * ref.y.abs(), "y")
    assert not y[:, :8].any()
    dx, dw, db = R.layer_norm_backward(gy, x, mean, rstd)
    assert dw is None and db is None
    (rx, ex), _, _ = ref.back(gy, 64)
    S.close(dx, rx, ex * 1.01 + S.F32 * rx.abs(), "grad_x")
    out = torch.empty((0, 24), device="cuda")
    assert R.layer_norm(out)[0].shape == (0, 24)
    w = torch.ones(24, device="cuda")
    _, dw, db = R.layer_norm_backward(out, out, mean[:0], rstd[:0], w, w)
    assert not dw.any() and not db.any()


def test_layer_norm_large_offset_keeps_the_variance(R):
    x = (torch.arange(64, device="cuda").float()[None] * 0.25 + 4096.0).repeat(3, 1)  # all exact in fp32
    y, mean, rstd = R.layer_norm(x)
    ref = S.Norm(x, None, None, 1e-5)
    S.close(rstd, ref.rstd, ref.rstd_err, "rstd")
    S.close(y, ref.y, ref.y_err, "y")


# ------------------------------------------------------------------ attention
def _offsets(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0)


def _bags(seed, B, q, k):
    g = torch.Generator()
    g.manual_seed(seed)
    ql = torch.randint(q[0], q[1] + 1, (B,), generator=g).tolist()
    kl = torch.randint(k[0], k[1] + 1, (B,), generator=g).tolist()
    return ql, kl


ATTEND = [
    # B, q lengths, k lengths, Hq, Hkv, D, share of masked keys
    (1, (1, 1), (1, 1), 1, 1, 8, 0.0),
    (8, (1, 4), (0, 50), 4, 4, 32, 0.0),
    (5, (1, 1), (900, 2100), 8, 2, 128, 0.0),
    (3, (1, 1), (300, 700), 16, 1, 64, 0.2),
    (7, (0, 16), (0, 300), 2, 2, 64, 0.1),
    (4, (17, 40), (100, 400), 6, 2, 72, 0.0),
    (2, (130, 260), (120, 390), 4, 4, 128, 0.05),
    (2, (128, 128), (128, 256), 2, 1, 64, 0.0),
    (3, (60, 90), (1, 140), 10, 2, 24, 0.3),
    (1, (513, 513), (1025, 1025), 3, 1, 96, 0.0),
    (1, (2, 2), (9000, 9000), 2, 1, 128, 0.0),
    (2, (3, 9), (60, 70), 130, 2, 16, 0.0),
    (6, (1, 200), (0, 500), 1, 1, 40, 1.0),
    (4, (70, 150), (0, 100), 2, 2, 64, 0.0),    # few keys, many rows
    (3, (100, 300), (1, 128), 6, 3, 128, 0.2),
    (5, (3, 40), (0, 90), 1, 1, 128, 0.1),      # few keys, few rows
    (9, (30, 64), (200, 260), 1, 1, 48, 0.0),
]


def _check_attend(R, seed, case, dtype, train=True, strided=False):
    B, ql, kl, Hq, Hkv, D, masked = case
    g = _gen(seed)
    ql, kl = _bags(seed, B, ql, kl)
    qo, ko = _offsets(ql), _offsets(kl)
    Tq, Tk, extra = sum(ql), sum(kl), 3  # rows behind the last bag
    if strided:  # q from heads-major memory, k and v halves of one row, out inside a wider row
        q = _randn((Hq, Tq + extra, D), dtype, g).transpose(0, 1)
        kv = _randn((Tk + extra, 2, Hkv, D), dtype, g)
        k, v = kv[:, 0], kv[:, 1]
        out = torch.full((Tq + extra, Hq, D + 8), 7.0, dtype=dtype, device="cuda")[:, :, 8:]
        dkv = torch.full_like(kv, 7.0)
        gk, gv = dkv[:, 0], dkv[:, 1]
    else:
        q, k, v = (_randn((n + extra, h, D), dtype, g) for n, h in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv)))
        out = torch.full((Tq + extra, Hq, D), 7.0, dtype=dtype, device="cuda")
        gk, gv = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    gq = torch.full_like(out, 7.0)
    grad = _randn((Tq + extra, Hq, D), dtype, g)
    lse = torch.full((Tq + extra, Hq), 7.0, device="cuda")
    mask = None
    if masked:
        mask = torch.rand(Tk + extra, device="cuda", generator=g) >= masked
    # what no bag and no unmasked key holds must not matter
    q[Tq:], k[Tk:], v[Tk:], grad[Tq:] = math.nan, math.inf, math.nan, math.inf
    if mask is not None:
        k[~mask], v[~mask] = math.nan, -math.inf
    scale = None if seed % 2 else 0.3
    mq, mk = max(ql + [1]), max(kl + [0]) + seed % 3
    R.attend(q, k, v, qo, ko, mq, mk, scale=scale, key_mask=mask, out=out, lse=lse)
    R.sequence_status_sync()
    sc = D ** -0.5 if scale is None else scale
    ref = S.attend(q[:Tq], k[:Tk], v[:Tk], qo, ko, sc, mask, grad[:Tq] if train else None)
    S.close(out[:Tq], *ref["out"], "out")
    S.close(lse[:Tq], *ref["lse"], "lse")
    assert (out[Tq:] == 7.0).all() and (lse[Tq:] == 7.0).all()
    if not train:
        return
    R.attend_backward(grad, q, k, v, out, lse, qo, ko, mq, mk, scale=scale, key_mask=mask, grad_q=gq, grad_k=gk,
                      grad_v=gv)
    R.sequence_status_sync()
    S.close(gq[:Tq], *ref["grad_q"], "grad_q")
    S.close(gk[:Tk], *ref["grad_k"], "grad_k")
    S.close(gv[:Tk], *ref["grad_v"], "grad_v")
    assert (gq[Tq:] == 7.0).all() and (gk[Tk:] == 7.0).all() and (gv[Tk:] == 7.0).all()
    first = [t.clone() for t in (gq, gk, gv)]
    R.attend_backward(grad, q, k, v, out, lse, qo, ko, mq, mk, scale=scale, key_mask=mask, grad_q=gq, grad_k=gk,
                      grad_v=gv)
    assert all(torch.equal(x[:n], y[:n]) for x, y, n in zip(first, (gq, gk, gv), (Tq, Tk, Tk)))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend(R, i, dtype):
    _check_attend(R, 100 + i, ATTEND[i], dtype)


@pytest.mark.parametrize("i", [1, 2, 4, 6, 9])
def test_attend_strided(R, i):
    _check_attend(R, 200 + i, ATTEND[i], BF16, strided=True)


@pytest.mark.parametrize("dtype,D,q", [(BF16, 64, 1), (F16, 64, 5), (BF16, 128, 1), (F16, 40, 16)])
def test_attend_of_few_rows_while_the_memory_is_busy(R, dtype, D, q):
    """Passes in a row over keys that L2 does not hold, beside copies: bit for bit
    what a pass by itself gives (and that is right)."""
    g = _gen(D + q)
    B = 100 * 64 // D
    ql, kl = _bags(D, B, (1, q), (1500, 5000))
    qo, ko = _offsets(ql), _offsets(kl)
    Q = _randn((sum(ql), 2, D), dtype, g)
    k, v = (_randn((sum(kl), 2, D), dtype, g) for _ in range(2))
    want = R.attend(Q, k, v, qo, ko, q, max(kl))
    torch.cuda.synchronize()
    some = slice(0, int(qo[4])), slice(0, int(ko[4]))
    ref = S.attend(Q[some[0]], k[some[1]], v[some[1]], qo[:5], ko[:5], D ** -0.5)
    S.close(want[0][some[0]], *ref["out"], "out")
    buf, side, got = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(side):
            for _ in range(3):
                buf[: 128 << 20].copy_(buf[128 << 20:])
        got.append(R.attend(Q, k, v, qo, ko, q, max(kl)))
    R.sequence_status_sync()
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,D,masked", [(BF16, 128, 0.0), (F16, 72, 0.1), (BF16, 64, 0.1)])
def test_attend_of_keys_and_values_that_arrive_late(R, dtype, D, masked):
    """Passes over different inputs in a row while copies keep the memory busy, so
    that a tile's values may still be on their way when the next tile's turn comes;
    most bags end inside a tile."""
    states = []
    for i in range(2):
        g = _gen(60 + i)
        ql, kl = _bags(60 + i, 12, (150, 300), (129, 1500))
        q, k, v = (_randn((sum(n), h, D), dtype, g) for n, h in ((ql, 4), (kl, 2), (kl, 2)))
        mask = torch.rand(sum(kl), device="cuda", generator=g) >= masked if masked else None
        qo, ko = _offsets(ql), _offsets(kl)
        ref = S.attend(q, k, v, qo, ko, D ** -0.5, mask)
        states.append(((q, k, v, qo, ko, max(ql), max(kl)), mask, ref))
    buf, side = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    got = []
    torch.cuda.synchronize()
    for i in range(24):
        with torch.cuda.stream(side):
            for _ in range(4):
                buf[: 128 << 20].copy_(buf[128 << 20:])
        a, mask, _ = states[i % 2]
        got.append(R.attend(*a, key_mask=mask))
    R.sequence_status_sync()
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        ref = states[i % 2][2]
        S.close(out, *ref["out"], f"out of pass {i}")
        S.close(lse, *ref["lse"], f"lse of pass {i}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,rows", [(1, 20), (3, 50), (5, 200)])
def test_attend_does_not_depend_on_rows_beside_it(R, Hq, rows, dtype):
    """A bag alone, before a bag of other queries, and after a call that leaves large
    values in shared memory: the same bits."""
    g = _gen(rows)
    q, k, v = (_randn((n, h, 64), dtype, g) for n, h in ((2 * rows, Hq), (1200, 1), (1200, 1)))
    q[rows:] *= 30
    alone = R.attend(q[:rows], k[:600], v[:600], _offsets([rows]), _offsets([600]), rows, 600)
    two = R.attend(q, k, v, _offsets([rows, rows]), _offsets([600, 600]), rows, 600)
    big = _randn((148 * 2 * 128, 1, 64), dtype, g, 60.0)
    R.attend(big, k[:128], v[:128], _offsets([big.shape[0]]), _offsets([128]), big.shape[0], 128)
    again = R.attend(q[:rows], k[:600], v[:600], _offsets([rows]), _offsets([600]), rows, 600)
    R.sequence_status_sync()
    for x, y, z in zip(alone, two, again):
        assert torch.equal(x, y[:rows]) and torch.equal(x, z)


def test_attend_large_scores(R):
    """Scores of thousands, of both signs: the running maximum carries them."""
    g = _gen(5)
    D = 64
    q, k, v = (_randn((n, 1, D), F16, g, m) for n, m in ((20, 30.0), (700, 30.0), (700, 1.0)))
    qo, ko = _offsets([20]), _offsets([700])
    out, lse = R.attend(q, k, v, qo, ko, 20, 700, scale=1.0)
    ref = S.attend(q, k, v, qo, ko, 1.0)
    S.close(out, *ref["out"], "out")
    S.close(lse, *ref["lse"], "lse")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [-0.7, 0.0])
@pytest.mark.parametrize("rows,keys,masked", [(9, 300, 0.1), (40, 100, 0.0), (150, 300, 0.1)])
def test_attend_negative_and_zero_scale(R, rows, keys, masked, scale, dtype):
    g = _gen(rows)
    q, grad = (_randn((rows, 2, 32), dtype, g) for _ in range(2))
    k, v = (_randn((keys, 1, 32), dtype, g) for _ in range(2))
    mask = torch.rand(keys, device="cuda", generator=g) >= masked
    k[~mask], v[~mask] = math.nan, math.inf
    qo, ko = _offsets([rows]), _offsets([keys])
    out, lse = R.attend(q, k, v, qo, ko, rows, keys, scale=scale, key_mask=mask)
    grads = R.attend_backward(grad, q, k, v, out, lse, qo, ko, rows, keys, scale=scale, key_mask=mask)
    R.sequence_status_sync()
    ref = S.attend(q, k, v, qo, ko, scale, mask, grad)
    for t, n in zip((out, lse, *grads), ("out", "lse", "grad_q", "grad_k", "grad_v")):
        S.close(t, *ref[n], n)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows", [1, 33])
def test_attend_of_many_short_bags(R, rows, dtype):
    """70000 bags of 3 keys, more than a grid's second dimension holds."""
    g = _gen(15)
    B, D = 70000, 16
    q, grad = (_randn((B * rows, 2, D), dtype, g) for _ in range(2))
    k, v = (_randn((B * 3, 2, D), dtype, g) for _ in range(2))
    qo, ko = (torch.arange(B + 1, device="cuda") * n for n in (rows, 3))
    out, lse = R.attend(q, k, v, qo, ko, rows, 3)
    gq, gk, gv = R.attend_backward(grad, q, k, v, out, lse, qo, ko, rows, 3)
    R.sequence_status_sync()
    for b in (0, 1, 32767, 65535, 65536, B - 1):
        a, c = slice(b * rows, (b + 1) * rows), slice(3 * b, 3 * b + 3)
        ref = S.attend(q[a], k[c], v[c], _offsets([rows]), _offsets([3]), 0.25, None, grad[a])
        for t, n in zip((out[a], lse[a], gq[a], gk[c], gv[c]), ("out", "lse", "grad_q", "grad_k", "grad_v")):
            S.close(t, *ref[n], n)


def test_attend_offsets_past_32_bits(R):
    """A cache whose last rows lie more than 2^32 elements in."""
    Tk, H, D = 1 << 20, 40, 128
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    kv = torch.zeros((2, Tk, H, D), dtype=BF16, device="cuda")
    g = _gen(6)
    n = 300
    kv[:, -n:] = _randn((2, n, H, D), BF16, g)
    q, grad = _randn((3, H, D), BF16, g), _randn((3, H, D), BF16, g)
    qo, ko = _offsets([0, 3]), torch.tensor([0, Tk - n, Tk], device="cuda")
    out, lse = R.attend(q, kv[0], kv[1], qo, ko, 3, Tk)
    small = S.attend(q, kv[0, -n:], kv[1, -n:], _offsets([3]), _offsets([n]), D ** -0.5, None, grad)
    S.close(out, *small["out"], "out")
    gk = torch.empty_like(kv)
    gq, _, _ = R.attend_backward(grad, q, kv[0], kv[1], out, lse, qo, ko, 3, Tk, grad_k=gk[0], grad_v=gk[1])
    R.sequence_status_sync()
    S.close(gq, *small["grad_q"], "grad_q")
    S.close(gk[0, -n:], *small["grad_k"], "grad_k")
    S.close(gk[1, -n:], *small["grad_v"], "grad_v")
    assert not gk[:, : Tk - n].any()  # keys of a bag without queries


def test_attend_reads_rows_in_any_order_of_strides(R):
    """Keys that share memory between heads' rows (a window over one buffer)."""
    g = _gen(11)
    buf = _randn((300 + 16, 32), F16, g)
    k = buf.as_strided((300, 2, 32), (32, 256, 1))  # head 1 is head 0, 8 rows on
    q = _randn((20, 2, 32), F16, g)
    qo, ko = _offsets([20]), _offsets([300])
    out, lse = R.attend(q, k, k, qo, ko, 20, 300)
    same, lse2 = R.attend(q, k.contiguous(), k.contiguous(), qo, ko, 20, 300)
    assert torch.equal(out, same) and torch.equal(lse, lse2)
    with pytest.raises(ValueError):  # but gradients need memory of their own
        R.attend_backward(out, q, k, k, out, lse, qo, ko, 20, 300, grad_k=buf.as_strided((300, 2, 32), (32, 256, 1)))


def test_attend_zeros_of_a_bag_of_keys_without_queries_past_32_bits(R):
    """2^27 keys of 128 in one bag without queries: 2^31 pieces of 16 bytes."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    n, B, D = 1 << 27, 444, 128  # bags enough that the keys are not split
    k = torch.zeros(8 * n + D, dtype=BF16, device="cuda").as_strided((n, 1, D), (8, D, 1))
    grad = torch.ones((n, 2, 1, D), dtype=BF16, device="cuda")
    q = torch.ones((1, 1, D), dtype=BF16, device="cuda")
    qo, ko = torch.zeros(B + 1, dtype=torch.int64, device="cuda"), _offsets([n] + [0] * (B - 1))
    R.attend_backward(q, q, k, k, q, torch.zeros((1, 1), device="cuda"), qo, ko, 1, n, grad_k=grad[:, 0],
                      grad_v=grad[:, 1])
    R.sequence_status_sync()
    assert not grad.any()


def test_attend_wide_bounds_need_no_join(R):
    """Bounds of 2^30 rows for 8 bags of a few: the blocks fit a grid, and nothing is joined."""
    g = _gen(13)
    q, k, v = (_randn((40, 1, 32), BF16, g) for _ in range(3))
    off = _offsets([5] * 8)
    out, lse = R.attend(q, k, v, off, off, 1 << 30, 5)
    R.sequence_status_sync()
    ref = S.attend(q, k, v, off, off, 32 ** -0.5)
    S.close(out, *ref["out"], "out")
    S.close(lse, *ref["lse"], "lse")


def test_status_of_calls_in_two_threads(R):
    """Two threads make calls that fail in different ways and ask for the status:
    a failure is reported to the thread that made it, or to the other one if that
    asked meanwhile."""
    g = _gen(14)
    w, bad = _randn((4, 8), F32, g), torch.tensor([9], device="cuda")
    q = _randn((4, 1, 16), BF16, g)
    good, long = _offsets([4]), _offsets([5])
    streams = [torch.cuda.Stream() for _ in range(2)]
    stop, reports = threading.Event(), []  # the other thread's: (from, to)

    def offsets_reported(stream):
        try:
            R.sequence_status_sync(stream)
        except R.RecisError as e:
            return "bag offsets" in str(e)
        return False

    def tokens():
        while not stop.is_set():
            R.embed_lookup(w, bad, stream=streams[0])
            t = time.monotonic()
            if offsets_reported(streams[0]):
                reports.append((t, time.monotonic()))

    R.attend(q, q, q, good, good, 4, 4)
    torch.cuda.synchronize()
    other = threading.Thread(target=tokens)
    other.start()
    open_calls = []
    for _ in range(2000):
        t = time.monotonic()
        R.attend(q, q, q, good, long, 4, 5, stream=streams[1])
        streams[1].synchronize()
        if not offsets_reported(streams[1]):
            open_calls.append((t, time.monotonic()))
    stop.set()
    other.join()
    offsets_reported(streams[0])
    lost = [c for c in open_calls if not any(r[0] <= c[1] and c[0] <= r[1] for r in reports)]
    assert not lost, f"{len(lost)} of 2000 failures were reported to no thread"


def test_attend_bad_offsets_are_reported(R):
    g = _gen(7)
    q, k, v = (_randn((40, 2, 32), BF16, g) for _ in range(3))
    good = _offsets([10, 30])
    for qo, ko, mq, mk in ((_offsets([10, 31]), good, 31, 30), (good, torch.tensor([0, 30, 20], device="cuda"), 30, 30),
                           (good, good, 29, 30), (good, good, 30, 20), (torch.tensor([-1, 10, 40], device="cuda"), good, 30, 30)):
        out, lse = R.attend(q, k, v, qo, ko, mq, mk)
        with pytest.raises(R.RecisError):
            R.sequence_status_sync()
        R.attend_backward(out, q, k, v, out, lse, qo, ko, mq, mk)
        with pytest.raises(R.RecisError):
            R.sequence_status_sync()
    R.attend(q, k, v, good, good, 30, 30)
    R.sequence_status_sync()


def test_attend_empty_calls(R):
    e = torch.empty((0, 2, 16), dtype=BF16, device="cuda")
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    out, lse = R.attend(e, e, e, none, none, 0, 0)
    assert out.shape == (0, 2, 16) and lse.shape == (0, 2)
    q = torch.ones((3, 2, 16), dtype=BF16, device="cuda")
    out, lse = R.attend(q, e, e, _offsets([1, 2]), _offsets([0, 0]), 2, 0)
    assert not out.any() and (lse == -math.inf).all()
    gq, gk, gv = R.attend_backward(q, q, e, e, out, lse, _offsets([1, 2]), _offsets([0, 0]), 2, 0)
    assert not gq.any() and gk.shape == (0, 2, 16)
    gq, gk, gv = R.attend_backward(e, e, q, q, e, lse[:0], _offsets([0, 0]), _offsets([1, 2]), 0, 2)
    assert not gk.any() and not gv.any()


@pytest.mark.parametrize("Hq", [2, 40, 128])
def test_attend_bounds_of_zero_are_bounds(R, Hq):
    """A bag of one row, or of one key, passes a bound of 0."""
    g = _gen(Hq)
    q, k = _randn((3, Hq, 16), F16, g), _randn((5, 1, 16), F16, g)
    one, none = _offsets([1, 2]), _offsets([0, 0])
    lse = torch.zeros((3, Hq), device="cuda")
    for qo, ko, mq, mk in ((_offsets([0, 1]), none, 0, 5), (none, _offsets([1, 0]), 3, 0), (one, _offsets([1, 0]), 2, 0)):
        R.attend(q, k, k, qo, ko, mq, mk)
        with pytest.raises(R.RecisError):
            R.sequence_status_sync()
        R.attend_backward(q, q, k, k, q, lse, qo, ko, mq, mk)
        with pytest.raises(R.RecisError):
            R.sequence_status_sync()
    R.attend(q, k, k, one, none, 2, 0)
    R.sequence_status_sync()


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (17, 1), (128, 1), (256, 2)])
def test_attend_rows_of_no_bag_with_a_bound_of_zero(R, Hq, Hkv):
    """max_q 0: no bag has queries, q's rows belong to none; keys get zeros."""
    g = _gen(Hq)
    D = 16
    q, k = _randn((3, Hq, D), BF16, g), _randn((700, Hkv, D), BF16, g)
    qo, ko = torch.zeros(3, dtype=torch.int64, device="cuda"), _offsets([650, 30])
    out, lse = torch.full_like(q, 7.0), torch.full((3, Hq), 7.0, device="cuda")
    R.attend(q, k, k, qo, ko, 0, 650, out=out, lse=lse)
    gq, gk, gv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    R.attend_backward(q, q, k, k, out, lse, qo, ko, 0, 650, grad_q=gq, grad_k=gk, grad_v=gv)
    R.sequence_status_sync()
    assert (out == 7.0).all() and (lse == 7.0).all() and (gq == 7.0).all()
    for t in (gk, gv):
        assert not t[:680].any() and (t[680:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,keys,D", [(5, 8, 64), (40, 100, 128), (150, 8, 128), (70, 128, 64)])
def test_attend_gradients_do_not_depend_on_neighbours(R, rows, keys, D, dtype):
    """A bag of few keys, alone and beside a bag of more than 128: the same bits."""
    g = _gen(rows + keys)
    ql, kl = [rows, 3, rows], [keys, 300, keys]
    q, grad = (_randn((sum(ql), 2, D), dtype, g) for _ in range(2))
    k, v = (_randn((sum(kl), 2, D), dtype, g) for _ in range(2))
    qo, ko = _offsets(ql), _offsets(kl)
    out, lse = R.attend(q, k, v, qo, ko, rows, 300)
    both = R.attend_backward(grad, q, k, v, out, lse, qo, ko, rows, 300)
    for i in (0, 2):
        a, b = slice(*qo[i:i + 2].tolist()), slice(*ko[i:i + 2].tolist())
        alone = R.attend_backward(grad[a], q[a], k[b], v[b], out[a], lse[a], _offsets([rows]), _offsets([keys]), rows,
                                  keys)
        for x, y, r in zip(both, alone, (a, b, b)):
            assert torch.equal(x[r], y)
    R.sequence_status_sync()


def _half_gradients(q, k, v, grad, scale):
    """The gradients of one bag and head in 64 bits with the errors that they may
    carry, [rows, D] each.  As sequence_ref.attend, but a term p or ds may be off by
    no subnormal step of fp16: the backward scales p by 2^14, and ds so that its
    bound, |grad| |v| + |delta| at their largest, is 2^13 or more."""
    Q, K, V, dO = (t.double() for t in (q, k, v, grad))
    D, n, u, step = Q.shape[1], K.shape[0], S.half_step(F16), S.least(F16)
    s = Q @ K.T * scale
    e = 2 * ((D + 4) * 2 * S.F32 * (Q.abs() @ K.abs().T) * abs(scale) + 4 * S.F32 * s.abs()).amax(
        1, keepdim=True) + (n + 64) * 2 * S.F32
    lse = torch.logsumexp(s, 1, keepdim=True)
    p = torch.exp(s - lse)
    o = p @ V
    o_err = (u + e) * (p @ V.abs()) + step * p.amax(1, keepdim=True) * V.abs().sum(0) + u * o.abs() + step
    dp, delta = dO @ V.T, (dO * o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    pe = p * (2 * e + 8 * S.F32 * lse.abs() + 2 * S.F32 * s.abs().amax(1, keepdim=True))
    delta_err = (dO.abs() * o_err).sum(1, keepdim=True) + (D + 2) * S.F32 * (dO * o).abs().sum(1, keepdim=True)
    dp_err = (D + 2) * 2 * S.F32 * (dO.abs() @ V.abs().T)
    bound = dO.norm(dim=1).max() * V.norm(dim=1).max() + (delta.abs() + delta_err).max()
    ds_err = pe * (dp - delta).abs() + p * (delta_err + dp_err) + (u + 4 * S.F32) * ds.abs() + step * 2.0 ** -13 * bound
    nq = (Q.shape[0] + 8) * 2 * S.F32
    gq, gk, gv = ds @ K * scale, ds.T @ Q * scale, p.T @ dO
    return ((gq, (ds_err + (n + 8) * 2 * S.F32 * ds.abs()) @ K.abs() * abs(scale) + (u + 4 * S.F32) * gq.abs() + step),
            (gk, (ds_err + nq * ds.abs()).T @ Q.abs() * abs(scale) + (u + 4 * S.F32) * gk.abs() + step),
            (gv, (pe + (u + nq) * p + step * 2.0 ** -14).T @ dO.abs() + (u + 4 * S.F32) * gv.abs() + step))


def _check_half_gradients(R, q, k, v, grad):
    qo, ko = _offsets([q.shape[0]]), _offsets([k.shape[0]])
    heads = [t[:, None].contiguous() for t in (q, k, v, grad)]
    out, lse = R.attend(*heads[:3], qo, ko, q.shape[0], k.shape[0], scale=0.125)
    got = R.attend_backward(heads[3], *heads[:3], out, lse, qo, ko, q.shape[0], k.shape[0], scale=0.125)
    R.sequence_status_sync()
    for x, (want, tol), name in zip(got, _half_gradients(q, k, v, grad, 0.125), ("grad_q", "grad_k", "grad_v")):
        # 65504 is fp16's largest number, and 65520 (half a step on) rounds to infinity
        want = torch.where(want.abs() - tol >= 65520, torch.copysign(torch.full_like(want, math.inf), want), want)
        S.close(x[:, 0], want, tol, name)


@pytest.mark.parametrize("rows,D", [(12, 64), (50, 128), (100, 64), (300, 128)])
@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-5])
def test_attend_half_gradients_of_long_bags(R, rows, D, size):
    """fp16, 6000 keys, gradients small enough for p (dp - delta) to be below the
    smallest normal number of fp16.  dp has the sign of a key's column of K, so that
    errors of ds add up in grad_q; q has columns that K lacks, for grad_k."""
    g = _gen(rows)
    n, h = 6000, D // 2
    sign = torch.where(torch.rand((n, 1), device="cuda", generator=g) < 0.5, -1.0, 1.0)
    pos = lambda m: torch.rand((m, D), device="cuda", generator=g) + 0.5  # noqa: E731
    q, k = _randn((rows, D), F32, g, 0.25), _randn((n, D), F32, g, 0.25)
    q[:, h:h + 8], k[:, h:h + 8] = 0.0, 4.0 * sign
    q[:, h + 8:], k[:, h + 8:] = 32.0, 0.0
    _check_half_gradients(R, *(t.to(F16) for t in (q, k, pos(n) * sign, pos(rows) * size)))


@pytest.mark.parametrize("rows,D", [(12, 64), (50, 128), (100, 64), (300, 128)])
def test_attend_half_gradients_of_keys_hardly_attended(R, rows, D):
    """fp16, half of 3000 keys with p about 2e-9 under gradients of thousands."""
    g = _gen(rows + 1)
    q, k, v = (_randn((m, D), F32, g, 0.25) for m in (rows, 3000, 3000))
    q[:, 0], k[:, 0] = 1.0, torch.where(torch.rand(3000, device="cuda", generator=g) < 0.5, -96.0, 0.0)
    grad = torch.rand((rows, D), device="cuda", generator=g) * 2000 + 1000
    _check_half_gradients(R, *(t.to(F16) for t in (q, k, v, grad)))


@pytest.mark.parametrize("rows,D", [(1, 64), (20, 64), (50, 128), (100, 64), (300, 128)])
@pytest.mark.parametrize("n", [2, 200])
def test_attend_half_gradients_with_ds_beyond_the_type(R, rows, D, n):
    """fp16, gradients of 10^4: ds of 2 keys passes 65504, grad_q and grad_k do not.
    The first 128 of 200 keys' are small, so that the scale of ds has to follow."""
    g = _gen(rows + 2)
    q, k, v, grad = (_randn((m, D), F32, g, x) for m, x in ((rows, 1e-4), (n, 1e-4), (n, 4.0), (rows, 8000.0)))
    if n > 128:
        v[:128] *= 1e-4
    _check_half_gradients(R, *(t.to(F16) for t in (q, k, v, grad)))


@pytest.mark.parametrize("rows", [3, 100])
def test_attend_half_gradients_beside_infinities(R, rows):
    """fp16: a row whose gradient holds an infinity spoils grad_k and grad_v of its
    bag, not grad_q of the other rows nor another bag."""
    g = _gen(rows + 3)
    q, grad = (_randn((2 * rows, 2, 64), F16, g) for _ in range(2))
    k, v = (_randn((800, 2, 64), F16, g) for _ in range(2))
    qo, ko = _offsets([rows, rows]), _offsets([400, 400])
    out, lse = R.attend(q, k, v, qo, ko, rows, 400)
    want = R.attend_backward(grad, q, k, v, out, lse, qo, ko, rows, 400)
    grad[1, 0, 5] = math.inf
    got = R.attend_backward(grad, q, k, v, out, lse, qo, ko, rows, 400)
    ref = S.attend(q, k, v, qo, ko, 0.125, None, grad.clamp(-65504, 65504))
    keep = torch.ones_like(q, dtype=torch.bool)
    keep[1, 0] = False
    S.close(got[0][keep], *(t[keep] for t in ref["grad_q"]), "grad_q")
    assert not torch.isfinite(got[0][1, 0]).any()
    assert torch.equal(got[0][rows:], want[0][rows:]) and torch.equal(got[0][:, 1], want[0][:, 1])
    for i in (1, 2):
        assert torch.equal(got[i][400:], want[i][400:]) and torch.equal(got[i][:, 1], want[i][:, 1])
        assert not torch.isfinite(got[i][:400, 0]).all()


# ------------------------------------------------------------------ differences
def test_gradients_against_differences(R):
    """Each gradient's product with a direction against the central difference
    of the 64-bit forward (its error is of the step's square and far below)."""
    g = _gen(9)
    x, gy = _randn((6, 24), F32, g), _randn((6, 24), F32, g)
    w, b = _randn((24,), F32, g), _randn((24,), F32, g)
    dirs = [_randn(t.shape, F32, g).double() for t in (x, w, b)]
    y, mean, rstd = R.layer_norm(x, w, b)
    grads = R.layer_norm_backward(gy, x, mean, rstd, w, b)
    h = 1e-4

    def norm(t):
        return (S.Norm(x.double() + t * dirs[0], w.double() + t * dirs[1], b.double() + t * dirs[2], 1e-5).y
                * gy.double()).sum()

    want = (norm(h) - norm(-h)) / (2 * h)
    got = sum((p.double() * d).sum() for p, d in zip(grads, dirs))
    mag = sum((p.double() * d).abs().sum() for p, d in zip(grads, dirs))
    assert abs(got - want) <= 400 * S.F32 * mag + 1e-5
    qo, ko = _offsets([3, 2]), _offsets([5, 40])
    q, k, v, go = (_randn((n, 2, 16), F16, g) for n in (5, 45, 45, 5))
    dirs = [_randn(t.shape, F32, g).double() for t in (q, k, v)]
    out, lse = R.attend(q, k, v, qo, ko, 3, 40)
    grads = R.attend_backward(go, q, k, v, out, lse, qo, ko, 3, 40)

    def att(t):
        ts = [p.double() + t * d for p, d in zip((q, k, v), dirs)]
        total = 0.0
        for i in range(2):
            for hd in range(2):
                Q, K, V = (p[a[i]:a[i + 1], hd] for p, a in zip(ts, (qo, ko, ko)))
                total = total + (torch.softmax(Q @ K.T * 0.25, 1) @ V * go.double()[qo[i]:qo[i + 1], hd]).sum()
        return total

    want = (att(h) - att(-h)) / (2 * h)
    tol = S.attend(q, k, v, qo, ko, 0.25, None, go)
    got = sum((p.double() * d).sum() for p, d in zip(grads, dirs))
    most = sum((tol[n][1] * d.abs()).sum() for n, d in zip(("grad_q", "grad_k", "grad_v"), dirs))
    assert abs(got - want) <= most + 1e-5
    t = torch.tensor([0, 2, 2, 1], device="cuda")
    grad = _randn((4, 8), F32, g)
    d = _randn((3, 8), F32, g).double()
    dw = R.embed_grad(t, grad, 3, scale=0.5)
    want = (S.lookup(d, t, 0.5, -1) * grad.double()).sum()  # the lookup is linear in the weight
    assert abs((dw.double() * d).sum() - want) <= 10 * S.F32 * (dw.double() * d).abs().sum() + 1e-6


# ------------------------------------------------------------------ streams, graphs
def _step(R, s):
    q = R.embed_lookup(s["w"], s["tok"], scale=2.0, out_dtype=BF16).view(-1, 4, 32)
    kv, mean, rstd = R.layer_norm(s["x"], s["g"], s["b"], out_dtype=BF16)
    k, v = kv[:, :64].unflatten(1, (2, 32)), kv[:, 64:].unflatten(1, (2, 32))
    bags = (s["qo"], s["ko"], s["mq"], s["mk"])
    out, lse = R.attend(q, k, v, *bags)
    dkv = torch.empty_like(kv)
    dq, _, _ = R.attend_backward(s["go"], q, k, v, out, lse, *bags, grad_k=dkv[:, :64].unflatten(1, (2, 32)),
                                 grad_v=dkv[:, 64:].unflatten(1, (2, 32)))
    dx, dg, db = R.layer_norm_backward(dkv, s["x"], mean, rstd, s["g"], s["b"])
    dw = R.embed_grad(s["tok"], dq.flatten(1), s["w"].shape[0], scale=2.0)
    return out, lse, dx, dg, db, dw


def _state(seed, ql=(3, 0, 40, 7), kl=(500, 9, 130, 0), V=50):
    g = _gen(seed)
    s = dict(w=_randn((V, 128), F32, g), x=_randn((sum(kl), 128), F32, g), g=_randn((128,), F32, g),
             b=_randn((128,), F32, g), go=_randn((sum(ql), 4, 32), BF16, g), qo=_offsets(ql), ko=_offsets(kl),
             mq=max(ql), mk=max(kl))
    s["tok"] = torch.randint(-1, V, (sum(ql),), device="cuda", generator=g)
    return s


def test_operators_together_captured_and_replayed(R):
    """The whole run captured twice (two graphs alive at once), replayed on new
    inputs in the captured buffers, against eager runs; and on another stream."""
    states = [_state(20), _state(21, (1, 1, 1, 1), (2000, 1, 64, 65), V=2000)]
    _step(R, states[0])  # the first call looks up the status word
    torch.cuda.synchronize()
    graphs = []
    for s in states:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = _step(R, s)
        graphs.append((gr, res))
    for k in range(2):
        for s in states:
            for n in ("w", "x", "g", "b", "go"):
                s[n].copy_(_randn(s[n].shape, s[n].dtype, _gen(30 + k)))
        want = [[t.clone() for t in _step(R, s)] for s in states]
        for gr, _ in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for (_, got), w in zip(graphs, want):
            assert all(torch.equal(p, q) for p, q in zip(got, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _step(R, states[0])
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    y = R.layer_norm(states[0]["x"], stream=side)[0]  # the stream as an argument
    side.synchronize()
    assert torch.equal(y, R.layer_norm(states[0]["x"])[0])
    R.sequence_status_sync()


@pytest.mark.parametrize("rows", [3, 150])
def test_attention_as_a_threads_first_call(R, rows):
    """A host thread that has made no CUDA call of its own has no context yet."""
    g = _gen(rows)
    q, k, v = (_randn((n, 2, 64), BF16, g) for n in (rows, 300, 300))
    bags = (_offsets([rows]), _offsets([300]), rows, 300)
    want = R.attend(q, k, v, *bags)
    want += R.attend_backward(q, q, k, v, *want, *bags)
    torch.cuda.synchronize()
    got, failed = {}, []

    def run(name, call):
        try:
            got[name] = call()
        except R.RecisError as e:
            failed.append((name, str(e)))

    for name, call in (("forward", lambda: R.attend(q, k, v, *bags)),
                       ("backward", lambda: R.attend_backward(q, q, k, v, *want[:2], *bags))):
        t = threading.Thread(target=run, args=(name, call))
        t.start()
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got["forward"] + got["backward"], want))


def test_calls_on_two_streams_at_once(R):
    states = [_state(40 + i) for i in range(4)]
    want = [_step(R, s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for _ in range(5):
        got = []
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                got.append(_step(R, s))
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(p, q))


# ------------------------------------------------------------------ attention pooling of a table
def test_sequence_attention_trains_the_table(R):
    """Two steps of the attention pooling against the 64-bit chain on the same
    rows: the answers, the dense gradients, and the table's rows after Adagrad
    with the chain's row gradients."""
    g = _gen(50)
    Hkv, Dh, Hq, V = 2, 16, 4, 30
    D = 2 * Hkv * Dh
    kw = dict(lr=0.05, adagrad_init_acc=0.5, init_scale=1.0, init_seed=3)
    table, plain = R.Table(D, R.ADAGRAD, **kw), R.Table(D, R.ADAGRAD, **kw)
    b0, b1 = R.Batch(), R.Batch()
    qw, nw, nb = _randn((V, Hq * Dh), F32, g), _randn((D,), F32, g) + 1, _randn((D,), F32, g)
    att = R.SequenceAttention(table, qw, Hq, Hkv, nw, nb, query_scale=1.5, dtype=F16)
    kl, ql = [40, 0, 7, 130], [2, 3, 0, 21]
    for step in range(2):
        keys = torch.randint(0, 60, (sum(kl),), device="cuda", generator=g) * 1009 + step
        tok = torch.randint(-1, V, (sum(ql),), device="cuda", generator=g)
        qo, ko = _offsets(ql), _offsets(kl)
        go = _randn((sum(ql), Hq, Dh), F16, g)
        mask = torch.rand(sum(kl), device="cuda", generator=g) < 0.9
        out = att.forward(b0, keys, ko, tok, qo, max(ql), max(kl), key_mask=mask)
        dquery, dnw, dnb = att.backward(go)
        table.status_sync()
        rows = torch.empty((sum(kl), D), device="cuda")
        plain.lookup_pooled(b1, keys, ko, 1, 4, unpooled_out=rows)
        # the chain in 64 bits, its 16-bit activations rounded where the kernels round them
        ref = S.Norm(rows, nw, nb, 1e-5)
        kv, q = ref.y.to(F16), S.lookup(qw, tok, 1.5, -1).to(F16).view(-1, Hq, Dh)
        k, v = kv[:, : D // 2].view(-1, Hkv, Dh), kv[:, D // 2:].view(-1, Hkv, Dh)
        a = S.attend(q, k, v, qo, ko, Dh ** -0.5, mask, go)
        # an input of the attention may round the other way (its fp32 value was next to a border): a step of
        # each input's type, 4 tolerances in all (those of q, k, v and the sums themselves)
        S.close(out, a["out"][0], 4 * a["out"][1] + 1e-4, "out")
        dkv, ekv = (torch.cat([a["grad_k"][i].flatten(1), a["grad_v"][i].flatten(1)], 1) for i in range(2))
        (dx, ex), (dw, ew), (db, eb) = ref.back(dkv, 64)
        S.close(dnb, db, eb + 4 * ekv.sum(0) + 1e-3, "norm bias")
        S.close(dnw, dw, ew + 4 * (ekv * ref.xh.abs()).sum(0) + 1e-3, "norm weight")
        wq, _ = S.embed_grad(tok, a["grad_q"][0].flatten(1), V, 1.5, -1)
        eq, _ = S.embed_grad(tok, a["grad_q"][1].flatten(1), V, 1.5, -1)
        S.close(dquery, wq, 4 * eq + 1e-4, "query weight")
        plain.backward_update(b1, grad_unpooled=dx.float())
        gk, ge, gs, _ = table.export()
        pk, pe, ps, _ = plain.export()
        assert (gk == pk).all()
        # a row moves by lr * g / (sqrt(acc) + eps), sqrt(acc) >= sqrt(0.5): 0.071 |dg| for a row's summed gradient,
        # whose terms are off by at most r (|e w| + mean|e w| + |xh| mean|e w xh|), e the attention's tolerance
        e = 4 * ekv * nw.double().abs()
        xh = ref.xh.abs()
        off = ref.rstd[:, None] * (e + e.mean(1, keepdim=True) + xh * (e * xh).mean(1, keepdim=True)) + ex
        per_key, _ = S.embed_grad(torch.searchsorted(torch.unique(keys), keys), off, torch.unique(keys).numel(), 1.0, -1)
        most = float(per_key.max()) * 0.071 * (step + 1) + 1e-5
        assert float(abs(ge - pe).max()) <= most
    for t in (table, plain, b0, b1):
        t.close()


def test_sequence_attention_gives_rows_of_no_bag_no_gradient(R):
    """A bag longer than max_keys, and tokens behind the last bag: as if the bag's
    keys were masked and the tokens were not there.  New memory is filled with NaN."""
    g = _gen(51)
    Hkv, Dh, Hq, V = 2, 16, 4, 30
    D = 2 * Hkv * Dh
    tables = [R.Table(D, R.ADAGRAD, lr=0.05, adagrad_init_acc=0.5, init_scale=1.0, init_seed=3) for _ in range(2)]
    batches = [R.Batch(), R.Batch()]
    qw, nw, nb = _randn((V, Hq * Dh), F32, g), _randn((D,), F32, g) + 1, _randn((D,), F32, g)
    kl, ql, tail = [40, 7, 140, 130], [2, 3, 4, 21], 5
    keys = torch.randint(0, 90, (sum(kl),), device="cuda", generator=g) * 1009
    tok = torch.randint(0, V, (sum(ql) + tail,), device="cuda", generator=g)
    qo, ko = _offsets(ql), _offsets(kl)
    go = _randn((sum(ql) + tail, Hq, Dh), F16, g)
    got = []
    torch.use_deterministic_algorithms(True, warn_only=True)  # fills new tensors with NaN
    try:
        for t, b, i in zip(tables, batches, range(2)):
            att = R.SequenceAttention(t, qw, Hq, Hkv, nw, nb, query_scale=1.5, dtype=F16)
            if i == 0:
                out = att.forward(b, keys, ko, tok, qo, max(ql), 135)
                with pytest.raises(R.RecisError):
                    R.sequence_status_sync()
                res = att.backward(go)
                with pytest.raises(R.RecisError):
                    R.sequence_status_sync()
            else:
                mask = torch.ones(sum(kl), dtype=torch.bool, device="cuda")
                mask[47:187] = False
                n = sum(ql)
                out = att.forward(b, keys, ko, tok[:n], qo, max(ql), 140, key_mask=mask)
                res = att.backward(go[:n])
                R.sequence_status_sync()
            t.status_sync()
            got.append((out, *res, *t.export()[:3]))
    finally:
        torch.use_deterministic_algorithms(False)
    n = sum(ql)
    assert not got[0][0][n:].any() and torch.equal(got[0][0][:n], got[1][0])
    for p, q in zip(got[0][1:4], got[1][1:4]):
        assert torch.isfinite(p).all() and torch.equal(p, q)
    for p, q in zip(got[0][4:], got[1][4:]):
        assert (p == q).all()
    for t in (*tables, *batches):
        t.close()


@pytest.mark.parametrize("kl,ql", [([0, 0], [2, 1]), ([3, 4], [0, 0]), ([0, 0], [0, 0]), ([5, 0], [0, 3]), ([], [])])
def test_sequence_attention_of_empty_bags(R, kl, ql):
    """Steps without keys, without tokens, without either, without bags."""
    g = _gen(52)
    table, batch = R.Table(64, R.ADAM, lr=0.05, init_scale=1.0, init_seed=3), R.Batch()
    w = torch.ones(64, device="cuda")
    att = R.SequenceAttention(table, _randn((30, 64), F32, g), 4, 2, w, w)
    keys = torch.arange(sum(kl), device="cuda") + 7
    tok = torch.randint(0, 30, (sum(ql),), device="cuda", generator=g)
    qo, ko = (torch.tensor([0] + n, device="cuda").cumsum(0) for n in (ql, kl))
    for _ in range(2):
        out = att.forward(batch, keys, ko, tok, qo, max(ql + [0]), max(kl + [0]))
        dquery, dnw, dnb = att.backward(_randn(out.shape, BF16, g))
        R.sequence_status_sync()
        table.status_sync()
        assert out.shape == (sum(ql), 4, 16) and dquery.shape == (30, 64)
        met = any(n and q for n, q in zip(kl, ql))  # a bag has both
        assert met == bool(out.any()) and all(met == bool(t.any()) for t in (dquery, dnw, dnb))
    assert table.size()[0] == sum(kl)
    table.close()
    batch.close()
