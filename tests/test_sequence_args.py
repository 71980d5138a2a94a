"""Refusals of the sequence operators on the host (no GPU): the C entry points
return RECIS_ERR_INVALID_ARG before they touch any array, the binding raises."""
import ctypes

import pytest
import torch

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def R():
    import recommender_sparse_embedding_b200 as R
    from recommender_sparse_embedding_b200 import build
    build.build()
    R.load()
    return R


P = 4096  # an address that no refused call reads


def _lookup(**kw):
    a = dict(w=P, wt=0, V=10, D=8, t=P, N=4, scale=1.0, pad=-1, out=P, ot=0, stride=8)
    a.update(kw)
    return [a["w"], a["wt"], a["V"], a["D"], a["t"], a["N"], a["scale"], a["pad"], a["out"], a["ot"], a["stride"], None]


@pytest.mark.parametrize("kw", [dict(w=None), dict(wt=3), dict(ot=-1), dict(V=0), dict(V=1 << 31), dict(D=0),
                                dict(D=65537), dict(N=-1), dict(N=1 << 31), dict(t=None), dict(out=None),
                                dict(stride=7), dict(w=P + 2), dict(t=P + 4), dict(out=P + 1, ot=1)])
def test_embed_lookup_refuses(R, kw):
    assert R.load().recis_embed_lookup(*_lookup(**kw)) == R.ERR_INVALID_ARG
    assert R.load().recis_last_error_string()


def _grad(**kw):
    a = dict(t=P, N=4, g=P, gt=1, gs=8, V=10, D=8, scale=1.0, pad=-1, acc=0, w=P, wt=0, ws=None, nb=0)
    a.update(kw)
    return [a[k] for k in ("t", "N", "g", "gt", "gs", "V", "D", "scale", "pad", "acc", "w", "wt", "ws", "nb")] + [None]


@pytest.mark.parametrize("kw", [dict(t=None), dict(g=None), dict(w=None), dict(gt=9), dict(wt=9), dict(gs=7),
                                dict(V=(1 << 31) - 1), dict(N=1 << 30), dict(acc=2), dict(g=P + 1), dict(w=P + 2),
                                dict(N=5000), dict(N=5000, ws=P, nb=100), dict(N=5000, ws=P + 16, nb=1 << 40)])
def test_embed_grad_refuses(R, kw):
    assert R.load().recis_embed_grad(*_grad(**kw)) == R.ERR_INVALID_ARG


def _norm(**kw):
    a = dict(x=P, xt=0, xs=8, M=4, D=8, w=P, b=P, wt=0, eps=1e-5, y=P, yt=1, ys=8, mean=P, rstd=P)
    a.update(kw)
    return [a[k] for k in ("x", "xt", "xs", "M", "D", "w", "b", "wt", "eps", "y", "yt", "ys", "mean", "rstd")] + [None]


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(xt=3), dict(yt=3), dict(wt=3), dict(xs=7), dict(ys=7),
                                dict(M=-1), dict(D=0), dict(eps=-1.0), dict(eps=float("nan")), dict(x=P + 2),
                                dict(mean=P + 2), dict(w=P + 1)])
def test_layer_norm_refuses(R, kw):
    assert R.load().recis_layer_norm(*_norm(**kw)) == R.ERR_INVALID_ARG


def _norm_back(**kw):
    a = dict(gy=P, yt=1, gs=8, x=P, xt=0, xs=8, M=4, D=8, w=P, wt=0, mean=P, rstd=P, gx=P, gxs=8, gw=P, gb=P, ws=P,
             nb=1 << 30)
    a.update(kw)
    return [a[k] for k in ("gy", "yt", "gs", "x", "xt", "xs", "M", "D", "w", "wt", "mean", "rstd", "gx", "gxs", "gw",
                           "gb", "ws", "nb")] + [None]


@pytest.mark.parametrize("kw", [dict(gy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(gs=7), dict(xs=7),
                                dict(gxs=7), dict(ws=None), dict(nb=8), dict(ws=P + 8), dict(gw=P + 2), dict(D=70000)])
def test_layer_norm_backward_refuses(R, kw):
    assert R.load().recis_layer_norm_backward(*_norm_back(**kw)) == R.ERR_INVALID_ARG


def _attend_args(**kw):
    from recommender_sparse_embedding_b200.sequence import AttendArgs
    a = AttendArgs(type=1, D=16, Hq=4, Hkv=2, B=1, Tq=3, Tk=5, max_q=3, max_k=5, scale=0.25, lse=P)
    for n in ("q_offsets", "k_offsets", "q", "k", "v", "out", "grad_out", "grad_q", "grad_k", "grad_v"):
        setattr(a, n, P)
    for n, H in (("q", 4), ("k", 2), ("v", 2), ("out", 4), ("grad_out", 4), ("grad_q", 4), ("grad_k", 2), ("grad_v", 2)):
        setattr(a, n + "_stride", 16 * H)
        setattr(a, n + "_head_stride", 16)
    for n, x in kw.items():
        setattr(a, n, x)
    return a


BAD_ATTEND = [dict(type=0), dict(type=3), dict(D=0), dict(D=12), dict(D=136), dict(Hkv=0), dict(Hq=3), dict(Hq=258),
              dict(B=-1), dict(Tq=1 << 31), dict(max_k=-1), dict(max_q=1 << 30), dict(scale=float("nan")), dict(q=None),
              dict(k=P + 8), dict(v_stride=36), dict(out=None), dict(lse=None), dict(lse=P + 2), dict(q_offsets=None),
              dict(k_offsets=P + 4), dict(k_head_stride=-8)]
BAD_BACK = [dict(grad_out=None), dict(grad_q=P + 8), dict(grad_k_stride=12), dict(grad_v=None)]


@pytest.mark.parametrize("kw", BAD_ATTEND)
def test_attend_refuses(R, kw):
    a = _attend_args(**kw)
    assert R.load().recis_attend(ctypes.byref(a), P, 1 << 40, None) == R.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_ATTEND + BAD_BACK)
def test_attend_backward_refuses(R, kw):
    a = _attend_args(**kw)
    assert R.load().recis_attend_backward(ctypes.byref(a), P, 1 << 40, None) == R.ERR_INVALID_ARG


def test_attend_workspace_is_asked_for(R):
    L, nb = R.load(), ctypes.c_int64()
    a = _attend_args(Tq=40, max_q=40)  # more rows than one tile: the backward keeps sums for them
    assert L.recis_attend_workspace(ctypes.byref(a), 1, ctypes.byref(nb)) == R.OK and nb.value > 0
    assert L.recis_attend_backward(ctypes.byref(a), P, nb.value - 1, None) == R.ERR_INVALID_ARG
    assert L.recis_attend_backward(ctypes.byref(a), P + 16, nb.value, None) == R.ERR_INVALID_ARG
    assert L.recis_attend_workspace(None, 0, ctypes.byref(nb)) == R.ERR_INVALID_ARG
    assert L.recis_attend_workspace(ctypes.byref(a), 0, None) == R.ERR_INVALID_ARG


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("Hq", [1, 16, 17, 64, 65, 128])
def test_attend_workspace_of_a_bound_of_zero(R, Hq, backward):
    """The launches take a bound of 0 as 1, so the workspace does too: rows of no
    bag (max_q 0) have their place in the backward's sums."""
    L, sizes = R.load(), []
    for bound in (0, 1):
        nb = ctypes.c_int64()
        a = _attend_args(Hq=Hq, Hkv=1, B=3, Tq=3, Tk=9000, max_q=bound, max_k=9000)
        assert L.recis_attend_workspace(ctypes.byref(a), backward, ctypes.byref(nb)) == R.OK
        sizes.append(nb.value)
    assert sizes[0] == sizes[1]
    if backward and Hq > 64:  # -delta and -lse of every row
        assert sizes[0] >= 2 * 3 * Hq * 4


def test_binding_refuses(R):
    w, t = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # no CPU fallback
        R.embed_lookup(w, t)
    with pytest.raises(TypeError):
        R.embed_lookup(w.double(), t)
    with pytest.raises(TypeError):
        R.embed_lookup(w, t.int())
    with pytest.raises(ValueError):
        R.embed_lookup(w.t(), t)
    with pytest.raises(ValueError):
        R.embed_grad(t, torch.zeros(4, 8), 4)
    with pytest.raises(ValueError):
        R.embed_grad(t, torch.zeros(3, 8), 4, accumulate=True)
    with pytest.raises(ValueError):  # rows share memory
        R.embed_grad(t, torch.zeros(1, 8).expand(3, 8), 4)
    with pytest.raises(ValueError):
        R.layer_norm(torch.zeros(8, 4).t())
    with pytest.raises(ValueError):
        R.layer_norm(torch.zeros(2, 8), torch.ones(7))
    with pytest.raises(TypeError):
        R.layer_norm(torch.zeros(2, 8), torch.ones(8), torch.ones(8, dtype=BF16))
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        R.layer_norm_backward(torch.zeros(2, 7), x, x[:, 0], x[:, 0])
    q = torch.zeros(4, 2, 16, dtype=BF16)
    o = torch.tensor([0, 4])
    with pytest.raises(TypeError):
        R.attend(q.float(), q.float(), q.float(), o, o, 4, 4)
    with pytest.raises(TypeError):
        R.attend(q, q.half(), q, o, o, 4, 4)
    with pytest.raises(ValueError):
        R.attend(q, q[:, :, :8], q[:, :, :8], o, o, 4, 4)
    with pytest.raises(ValueError):
        R.attend(q, q, q[:3], o, o, 4, 4)
    with pytest.raises(ValueError):
        R.attend(q, q, q, o, o[:1], 4, 4)
    with pytest.raises(ValueError):
        R.attend(q, q, q, o, o, 4, 4, key_mask=torch.ones(3, dtype=torch.bool))
    with pytest.raises(TypeError):
        R.attend(q, q, q, o.int(), o, 4, 4)


def test_outputs_whose_rows_share_memory_are_refused():
    from recommender_sparse_embedding_b200.sequence import _written
    base = torch.zeros(4, 2, 16, dtype=BF16)
    _written(base, "t", (32, 16))
    _written(base.transpose(0, 1), "t", (16, 32))
    for bad in ((0, 16), (16, 16), (32, 0), (8, 64)):
        with pytest.raises(ValueError):
            _written(base, "t", bad)


def test_sequence_attention_refuses_rows_that_do_not_fit(R):
    class T:
        dim = 64
    w = torch.ones(64)
    with pytest.raises(ValueError):
        R.SequenceAttention(T(), torch.zeros(5, 64), 4, 3, w, w)
    with pytest.raises(ValueError):
        R.SequenceAttention(T(), torch.zeros(5, 60), 4, 2, w, w)
    assert R.SequenceAttention(T(), torch.zeros(5, 64), 4, 2, w, w).head_dim == 16
    with pytest.raises(RuntimeError):
        R.SequenceAttention(T(), torch.zeros(5, 64), 4, 2, w, w).backward(w)


def test_sequence_attention_looks_at_the_device_first(R):
    """Tensors that are not on one GPU are refused before the table sees them, which
    takes its stream from the current device."""
    class T:
        dim = 64

        def lookup_pooled(self, *a, **kw):
            raise AssertionError("the lookup ran")

    w, n, o = torch.ones(64), torch.zeros(3, dtype=torch.int64), torch.tensor([0, 3])
    att = R.SequenceAttention(T(), torch.zeros(5, 64), 4, 2, w, w)
    with pytest.raises(ValueError):
        att.forward(None, n, o, n, o, 3, 3)


def test_rows_of_views():
    from recommender_sparse_embedding_b200.sequence import _rows
    x = torch.zeros(4, 6, 10)
    assert _rows(x, "x") == (24, 10, 10)
    assert _rows(x[:, :, 2:7], "x") == (24, 5, 10)
    assert _rows(x[:, 1], "x") == (4, 10, 60)
    assert _rows(x[1:2, 3:4, :4], "x") == (1, 4, 4)
    assert _rows(x[:0], "x")[0] == 0
    for bad in (x[:, :3], x.transpose(0, 1), x[:, :, ::2], x[:, :, :1].expand(4, 6, 3), x[:1].expand(3, 6, 10)):
        with pytest.raises(ValueError):
            _rows(bad, "x")
    with pytest.raises(ValueError):
        _rows(x, "x", 9)
