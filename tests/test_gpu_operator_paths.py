"""The kernels of the training-step operators that large shapes and mixed layouts take, at
sizes a test can afford: each way of summing a table gradient (accesses of 8, 2 and 1
elements, one to four passes of the sort, one to eight groups of the join), layer norm of rows
held by a block over many turns and of matrices that no common cut fits, and clipping by
several launches. Bounds as derived in test_gpu_operators.py, whose helpers these tests use.
"""
import numpy as np
import pytest
import torch

import vision_language_projector_b200 as vp
from oracle import operators as P
from test_gpu_operators import BF, HF, PAIRS, SF, TOKEN, U, _f64, _half, _ids, _ln_bounds, _place, _rand, _within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ table gradient
def _check_table_gradient(ids, d_out, vocab, layout="dense", scale=float(np.float32(0.3))):
    n, N = len(ids), d_out.shape[1]
    d_dev = _place(d_out, layout)
    want, mag = P.embed_backward(ids.numpy(), _f64(d_out), vocab, scale, TOKEN)
    inside = ids[(ids != TOKEN) & (ids >= 0) & (ids < vocab)].numpy()
    m = int(np.bincount(inside, minlength=1).max()) if len(inside) else 0
    bad = len(inside) < int((ids != TOKEN).sum())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _place(torch.full((vocab, N), float("nan")), layout)
    vp.embed_backward(ids.cuda(), d_dev, got, scale=scale, image_token_id=TOKEN, status=status)
    _within(got, want, (m + 3) * U * mag, "sums")
    assert int(status) == (vp.ERR_INVALID_ARG if bad else vp.OK)
    base = _rand((vocab, N), SF, 6)
    acc = _place(base, layout)
    status.zero_()
    vp.embed_backward(ids.cuda(), d_dev, acc, scale=scale, image_token_id=TOKEN, accumulate=True, status=status)
    _within(acc, _f64(base) + want, (m + 3) * U * (mag + np.abs(_f64(base))), "accumulated")
    assert torch.equal(acc.cpu()[mag.sum(1) == 0], base[mag.sum(1) == 0])
    assert int(status) == (vp.ERR_INVALID_ARG if bad else vp.OK)
    again = _place(torch.full((vocab, N), float("nan")), layout)
    vp.embed_backward(ids.cuda(), d_dev, again, scale=scale, image_token_id=TOKEN)
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("kind", ["rank", "one"])
@pytest.mark.parametrize("n,N,layout", [(5000, 34, "dense"), (5000, 130, "dense"), (5000, 578, "dense"), (3000, 1002, "dense"),
                                        (3000, 2048, "dense"), (3000, 2058, "dense"), (2500, 2560, "padded"),
                                        (2500, 4096, "dense"), (3000, 601, "dense"), (3000, 1501, "odd"),
                                        (2500, 2561, "shifted"), (300, 34, "dense"), (300, 578, "dense"),
                                        (2048, 1026, "padded"), (2048, 64, "dense")])
def test_table_gradient_by_every_access_and_join(dtype, kind, n, N, layout):
    vocab = 60
    d_out = _rand((n, N), dtype, 5)
    _check_table_gradient(_ids(kind, n, vocab, 4), d_out, vocab, layout)


@pytest.mark.parametrize("n", [300, 5000])
@pytest.mark.parametrize("N", [8, 34, 7])
def test_table_gradient_accumulates_past_bad_ids(n, N):
    ids = _ids("rank", n, 40, 9)
    ids[::7], ids[3::11], ids[5::13], ids[6::17] = 40, -1, 1 << 40, TOKEN
    _check_table_gradient(ids, _rand((n, N), BF, 10), 40)


@pytest.mark.parametrize("vocab", [(1 << 10) - 1, 1 << 10, (1 << 20) - 1, (1 << 20) + 5])
def test_table_gradient_sorts_in_one_to_three_passes(vocab):
    """Keys go up to vocab itself (rows that count for nothing): 10, 11, 20 and 21 bits."""
    n = 5000
    ids = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(11))
    ids[:1500], ids[1500:1600], ids[2000:2500] = vocab - 1, 0, TOKEN
    ids[2500:2600] = torch.arange(100) * (vocab // 100)
    _check_table_gradient(ids, _rand((n, 8), BF, 12), vocab)


def test_table_gradient_sorts_in_four_passes():
    """31 bits of key, and a table of more than 2^32 bytes."""
    n, vocab = 3000, (1 << 30) + 7
    ids = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(13))
    ids[::3], ids[1::3] = vocab - 1, torch.arange(1000) << 20
    d_out = _rand((n, 1), SF, 14)
    got = torch.full((vocab, 1), float("nan"), device="cuda")
    vp.embed_backward(ids.cuda(), d_out.cuda(), got)
    seen, where = np.unique(ids.numpy(), return_inverse=True)
    want, mag = np.zeros((len(seen), 1)), np.zeros((len(seen), 1))
    np.add.at(want, where, _f64(d_out))
    np.add.at(mag, where, np.abs(_f64(d_out)))
    rows = torch.from_numpy(seen).cuda()
    _within(got[rows], want, 1003 * U * mag)
    got[rows] = 0
    assert int(torch.count_nonzero(got)) == 0


# ------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("rows,C,lx,ly", [(40, 257, "dense", "shifted"), (900, 257, "shifted", "dense"), (700, 1000, "odd", "dense"),
                                          (300, 1152, "dense", "odd"), (5, 5120, "shifted", "padded"), (700, 6144, "dense", "padded"),
                                          (400, 7168, "padded", "dense"), (300, 7618, "dense", "dense"), (200, 9216, "dense", "dense"),
                                          (170, 14336, "dense", "dense"), (7, 30000, "dense", "dense"), (3, 57344, "padded", "dense"),
                                          (200, 2560, "dense", "dense"), (160, 5119, "dense", "dense")])
def test_layernorm_of_long_rows_and_mixed_layouts(pair, rows, C, lx, ly):
    tx, ty = pair
    x = _rand((rows, C), tx, 10, 2.0, 0.5)
    gamma, beta = _rand((C,), SF, 11, 0.3, 1.0), _rand((C,), SF, 12, 0.2)
    y = _place(torch.full((rows, C), float("nan"), dtype=ty), ly)
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    vp.layernorm(_place(x, lx), y, gamma.cuda(), beta.cuda(), 1e-5, mean, rstd)
    want, m, r = P.layernorm(_f64(x), _f64(gamma), _f64(beta), float(np.float32(1e-5)))
    by, bm, br = _ln_bounds(_f64(x), _f64(gamma), _f64(beta), m, r, want, ty)
    _within(mean, m, bm, "mean")
    _within(rstd, r, br + U * r, "rstd")
    _within(y, want, by, "y")


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("rows,C,lx,ldy,ldx", [(3000, 2048, "dense", "dense", "dense"), (2500, 5120, "dense", "dense", "dense"),
                                               (1500, 4097, "dense", "dense", "dense"), (900, 8192, "padded", "dense", "padded"),
                                               (700, 9216, "dense", "dense", "dense"), (600, 14336, "dense", "dense", "dense"),
                                               (40, 257, "dense", "shifted", "odd"), (3000, 257, "dense", "shifted", "odd"),
                                               (512, 256, "shifted", "dense", "padded"), (513, 256, "shifted", "dense", "padded"),
                                               (700, 1001, "odd", "dense", "shifted"), (1, 8000, "dense", "shifted", "dense"),
                                               (600, 16392, "dense", "dense", "dense")])
def test_layernorm_backward_of_long_rows_and_mixed_layouts(pair, rows, C, lx, ldy, ldx):
    tx, ty = pair
    x, d_y, gamma = _rand((rows, C), tx, 20, 2.0, 0.5), _rand((rows, C), ty, 21), _rand((C,), SF, 22, 0.3, 1.0)
    _, mean, rstd = P.layernorm(_f64(x))
    mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
    x64, dy64, g64, m64, r64 = (_f64(t) for t in (x, d_y, gamma, mean, rstd))
    want_dx, want_dg, want_db = P.layernorm_backward(x64, m64, r64, dy64, g64)
    xhat, g = (x64 - m64[:, None]) * r64[:, None], dy64 * g64
    D, (h, t) = C / 32 + 64, _half(tx)
    mg, mgx = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    bdx = (r64[:, None] * (3 * U * np.abs(g) + (D + 3) * U * mg + np.abs(xhat) * (D + 8) * U * mgx
                           + 6 * U * np.abs(xhat) * np.abs((g * xhat).mean(1, keepdims=True)))
           + (4 * U + h) * np.abs(want_dx) + t)
    bdg, bdb = (rows + 8) * U * np.abs(dy64 * xhat).sum(0), (rows + 8) * U * np.abs(dy64).sum(0)
    dx = _place(torch.full((rows, C), float("nan"), dtype=tx), ldx)
    dg, db, dg1 = (torch.full((C,), float("nan"), device="cuda") for _ in range(3))
    args = (_place(x, lx), mean.cuda(), rstd.cuda(), _place(d_y, ldy), gamma.cuda())
    work = torch.full((max(1, vp.layernorm_backward_workspace(rows, C)),), 255, dtype=torch.uint8, device="cuda")
    vp.layernorm_backward(*args, dx, dg, db, workspace=work)
    _within(dx, want_dx, bdx, "d_x")
    _within(dg, want_dg, bdg, "d_gamma")
    _within(db, want_db, bdb, "d_beta")
    vp.layernorm_backward(*args, d_gamma=dg1)
    _within(dg1, want_dg, bdg, "d_gamma alone")


# ------------------------------------------------------------------ clipping by several launches
SEVERAL = [[300_000, 77], [40_000] * 7, [999] * 20, [5] * 900 + [70_001]]


@pytest.mark.parametrize("sizes", SEVERAL)
def test_clip_by_several_launches_of_extreme_values(sizes):
    for scale in (1e25, 1e-30, 1e-38):
        ts = [_rand((n,), SF, 40 + i, scale).cuda() for i, n in enumerate(sizes)]
        norm = torch.empty(1, device="cuda")
        out = [torch.empty_like(t) for t in ts]
        work = torch.full((vp.clip_grads_workspace(len(ts)),), 255, dtype=torch.uint8, device="cuda")
        vp.clip_grads(ts, scale, norm, out, workspace=work)
        want_norm, want = P.clip_grads([_f64(t) for t in ts], scale)
        _within(norm, np.array([want_norm]), 8 * U * want_norm + 2.0 ** -150)
        for t, w in zip(out, want):
            _within(t, w, np.abs(w) * 12 * U + 2.0 ** -150)
    # a coefficient below fp32's normal range
    ts = [torch.full((n,), 3e38, device="cuda") for n in sizes]
    out = [torch.empty_like(t) for t in ts]
    vp.clip_grads(ts, 1e-3, None, out)
    for o, w in zip(out, P.clip_grads([_f64(t) for t in ts], 1e-3)[1]):
        _within(o, w, np.abs(w) * 12 * U + 2.0 ** -150)


@pytest.mark.parametrize("sizes", SEVERAL)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_by_several_launches_of_infinities_and_nan(sizes, bad):
    ts = [torch.ones(n, device="cuda", dtype=(SF, BF)[i % 2]) for i, n in enumerate(sizes)]
    ts[0][sizes[0] // 2] = bad
    norm = torch.empty(1, device="cuda")
    want_norm, want = P.clip_grads([_f64(t) for t in ts], 1.0)
    vp.clip_grads(ts, 1.0, norm)
    np.testing.assert_array_equal(_f64(norm), [want_norm])
    for t, w in zip(ts, want):
        np.testing.assert_array_equal(_f64(t), w)


@pytest.mark.parametrize("sizes", SEVERAL)
def test_clip_by_several_launches_on_streams_and_in_graphs(sizes):
    def grads(seed):
        return [_rand((n,), (SF, BF, HF)[i % 3], seed + i).cuda() for i, n in enumerate(sizes)]

    def outputs(ts):
        return [torch.zeros_like(t) for t in ts], torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")

    def run(ts, o, stream=None):
        vp.clip_grads(ts, 0.5, o[1], o[0], stream=stream)
        vp.grad_norm(ts, o[2], stream=stream)

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])

    ins = [grads(500), grads(9500)]
    want = []
    for ts in ins:
        want.append(outputs(ts))
        run(ts, want[-1])
        assert torch.equal(want[-1][1], want[-1][2])
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [outputs(ts) for ts in ins]
    torch.cuda.synchronize()
    for _ in range(10):
        for ts, o, s in zip(ins, got, streams):
            run(ts, o, s)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))
    graphs, got, held = [], [outputs(ts) for ts in ins], [[t.clone() for t in ts] for ts in ins]
    for ts, o in zip(held, got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(ts, o)
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for k, ts in enumerate(held):
            for dst, src in zip(ts, ins[order[k]]):
                dst.copy_(src)
        torch.cuda.synchronize()
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(same(o, want[order[k]]) for k, o in enumerate(got))
