"""The training-step operators on a B200 against their fp64 definitions.

Tolerances, with u = 2^-24 (fp32's half step, relative) and h = finfo(type).eps / 2 for the
one rounding of a result to its type (plus half the smallest subnormal of that type, t):

lookup       one fp32 product, one rounding: |v| (h + u) + t.
table grad   a sum of m fp32 terms in any order is off by at most (m - 1) u times the sum of
             |terms| to first order; scaling and the final add round twice: (m + 3) u mag.
layer norm   the kernels add a row's C elements in chains of at most D = C / 32 + 64 (each of
             at least 32 lanes, or one chain of up to 64, then a tree of 16 steps at most):
             |d_mean| <= (D + 2) u mean|x|; the variance about that mean is off by d_mean^2
             and (D + 4) u relative, so rstd by R = (D + 4) u + d_mean^2 rstd^2 / 2 + 4 u
             relative; y = (x - mean) rstd gamma + beta then by
             |gamma| rstd (|d_mean| + u |x - mean|) + |xhat gamma| (R + 4 u) + u |y| + h |y| + t.
its gradients  given the statistics, xhat rounds twice; the two row means round their chains:
             rstd (3 u |g| + (D + 3) u mean|g| + |xhat| (D + 8) u mean|g xhat|
             + 6 u |xhat mean(g xhat)|) + (4 u + h) |d_x| + t; column sums of R rows: (R + 8) u
             times the sum of |terms|.
clip         squares and sums of 8 in fp32, the rest in fp64: the norm within 8 u relative;
             a clipped value |v| (h + 11 u) + t.
All bounds get a factor 1.01 for the second-order terms.
"""
import numpy as np
import pytest
import torch

import vision_language_projector_b200 as vp
from oracle import operators as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TOKEN = 100015
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(BF, BF), (HF, HF), (SF, SF), (SF, BF), (SF, HF)]


def _half(dtype):
    f = torch.finfo(dtype)
    # half a step, and half the smallest subnormal, of the type
    return f.eps / 2, f.smallest_normal * f.eps / 2


def _rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, want, bound, what=""):
    err = np.abs(_f64(got) - want)
    assert np.isfinite(err).all(), what
    assert (err <= 1.01 * bound + 1e-300).all(), f"{what}: {np.max(err - 1.01 * bound)} over, err {err.max()}"


def _place(t, layout):
    """A CUDA copy of the matrix t: "dense", "padded" (rows 16-byte aligned, a gap between
    them), "odd" (rows of odd distance) or "shifted" (dense, one element off alignment)."""
    r, c = t.shape
    if layout == "dense":
        return t.cuda()
    if layout == "shifted":
        flat = torch.zeros(r * c + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(r, c)
    ld = -(-c // 8) * 8 + 16 if layout == "padded" else c + 3 - c % 2
    big = torch.full((r, ld), 77.0, dtype=t.dtype, device="cuda")
    big[:, :c] = t.cuda()
    return big[:, :c]


LAYOUTS = ["dense", "padded", "odd", "shifted"]


# ------------------------------------------------------------------ lookup
@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("n,N,vocab,layout", [(1, 1, 1, "dense"), (7, 64, 50, "padded"), (33, 1000, 50, "dense"),
                                              (65, 1001, 300, "dense"), (130, 77, 300, "odd"), (12, 520, 9, "shifted"),
                                              (200, 128, 1000, "dense"), (5, 5120, 40, "dense"), (700, 9, 3, "padded")])
def test_embed(pair, n, N, vocab, layout):
    ti, to = pair
    table, out = _rand((vocab, N), ti, 1), _rand((n + 2, N), to, 2)
    ids = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(3))
    ids[n // 3:n // 2] = TOKEN
    scale = float(np.float32(1.7))
    got = _place(out, layout)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vp.embed(ids.cuda(), _place(table, layout), got, scale=scale, image_token_id=TOKEN, status=status)
    want = P.embed(ids.numpy(), _f64(table), _f64(out), scale, TOKEN)
    h, t = _half(to)
    _within(got, want, np.abs(want) * (h + U) + t)
    stay = np.r_[np.arange(n)[ids.numpy() == TOKEN], n, n + 1]
    assert torch.equal(got.cpu()[stay], out[stay])                 # placeholders, and rows past the ids
    assert int(status) == vp.OK
    if layout in ("padded", "odd"):
        assert (got._base[:, N:] == 77).all()                      # the gaps between the rows


def test_embed_copies_bits_at_scale_one():
    for dtype, bits in ((BF, torch.int16), (HF, torch.int16), (SF, torch.int32)):
        table = torch.randint(-2 ** 15, 2 ** 15, (6, 40), dtype=bits).cuda().view(dtype)      # NaN patterns too
        out = torch.zeros(6, 40, dtype=dtype, device="cuda")
        vp.embed(torch.arange(6).cuda(), table, out)
        assert torch.equal(out.view(bits), table.view(bits))


def test_embed_bad_ids():
    table, out = _rand((10, 24), BF, 1).cuda(), torch.ones(6, 24, dtype=BF, device="cuda")
    ids = torch.tensor([0, -1, 10, -200, 1 << 40, 9]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vp.embed(ids, table, out, image_token_id=-200, status=status)      # a negative placeholder id is a placeholder
    assert int(status) == vp.ERR_INVALID_ARG
    assert (out[[1, 2, 4]] == 0).all() and (out[3] == 1).all() and torch.equal(out[5], table[9])
    status.fill_(vp.ERR_TIMEOUT)
    vp.embed(ids, table, out, status=status)
    assert int(status) == vp.ERR_TIMEOUT                               # the first error stays
    vp.embed(ids, table, out)                                          # no status wanted
    d_table = torch.empty(10, 24, device="cuda")
    status.zero_()
    vp.embed_backward(ids, out, d_table, status=status)
    assert int(status) == vp.ERR_INVALID_ARG
    want, mag = P.embed_backward(ids.cpu().numpy(), _f64(out), 10)
    _within(d_table, want, 4 * U * mag)


def test_lookup_beyond_32_bit_offsets():
    """Rows past 2^31 elements of the table, and past 2^32 bytes of its gradient."""
    N, vocab = 4096, 600_000
    table = torch.empty(vocab, N, dtype=BF, device="cuda")
    rows = torch.tensor([vocab - 1, 524_288, 524_287, 0]).cuda()
    table[rows] = _rand((4, N), BF, 1).cuda()
    out = torch.empty(4, N, dtype=BF, device="cuda")
    vp.embed(rows, table, out)
    assert torch.equal(out, table[rows])
    del table
    d_table = torch.full((vocab, N), float("nan"), device="cuda")
    vp.embed_backward(rows, out, d_table, scale=2.0)
    assert torch.equal(d_table[rows], out.float() * 2)
    assert int(torch.count_nonzero(d_table)) == int(torch.count_nonzero(out))       # and zeros in every other place
    assert not torch.isnan(d_table[-3:]).any()


# ------------------------------------------------------------------ table gradient
def _ids(kind, n, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "rank":
        ids = torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * np.log(vocab + 1)).sub(1).floor().long()
        return ids.clamp(0, vocab - 1)
    if kind == "one":
        return torch.full((n,), vocab // 2, dtype=torch.int64)
    if kind == "none":
        return torch.full((n,), TOKEN, dtype=torch.int64)
    if kind == "down":
        return torch.arange(n - 1, -1, -1) % vocab
    ids = torch.randint(0, vocab, (n,), generator=g)
    ids[n // 4:3 * n // 4] = TOKEN
    return ids


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("kind,n,N,vocab,layout",
                         [("mixed", 1, 8, 1, "dense"), ("mixed", 200, 128, 1000, "dense"), ("rank", 3000, 40, 50, "padded"),
                          ("one", 5000, 24, 7, "dense"), ("none", 300, 64, 20, "dense"), ("down", 1023, 33, 1024, "odd"),
                          ("rank", 1025, 1001, 70, "dense"), ("mixed", 4097, 136, 3000, "shifted"),
                          ("rank", 20000, 16, 102400, "dense"), ("down", 2049, 1040, 2048, "dense"),
                          ("one", 131, 2056, 3, "padded"), ("mixed", 64, 5, 2, "dense")])
def test_embed_backward(dtype, kind, n, N, vocab, layout):
    ids = _ids(kind, n, vocab, 4)
    d_out = _rand((n + 1, N), dtype, 5)
    d_out[n:] = float("nan")                                           # past the ids: not read
    if vocab > 1:
        d_out[:n][(ids == TOKEN)] = float("nan")                       # placeholders: not read
    scale = float(np.float32(0.3))
    d_dev = _place(d_out, layout)
    clean = torch.nan_to_num(d_out.float()).double().numpy()
    want, mag = P.embed_backward(ids.numpy(), clean, vocab, scale, TOKEN)
    m = int(np.bincount(ids[ids != TOKEN].numpy(), minlength=1).max()) if (ids != TOKEN).any() else 0
    got = _place(torch.full((vocab, N), float("nan")), layout)
    vp.embed_backward(ids.cuda(), d_dev, got, scale=scale, image_token_id=TOKEN)
    _within(got, want, (m + 3) * U * mag)
    base = _rand((vocab, N), SF, 6)
    acc = _place(base, layout)
    vp.embed_backward(ids.cuda(), d_dev, acc, scale=scale, image_token_id=TOKEN, accumulate=True)
    _within(acc, _f64(base) + want, (m + 3) * U * (mag + np.abs(_f64(base))))
    absent = torch.from_numpy(mag.sum(1) == 0)
    assert torch.equal(acc.cpu()[absent], base[absent])
    if layout in ("padded", "odd"):
        assert (acc._base[:, N:] == 77).all()
    again = torch.empty(vocab, N, device="cuda")
    vp.embed_backward(ids.cuda(), d_dev, again, scale=scale, image_token_id=TOKEN)
    assert torch.equal(again, got)                                     # a fixed order


def test_embed_backward_heavy_token_order_and_size():
    """300,000 rows of two tokens: many passes' worth of rows for one sum."""
    n, N = 300_000, 72
    ids = (torch.arange(n) % 7 == 0).long() * 99_999
    d_out = _rand((n, N), BF, 8)
    got = torch.empty(100_000, N, device="cuda")
    vp.embed_backward(ids.cuda(), d_out.cuda(), got)
    d64 = _f64(d_out)
    for t in (0, 99_999):
        rows = d64[ids.numpy() == t]
        # chunks of at most 128 rows in fp32, their sums in fp64
        _within(got[t], rows.sum(0), 130 * U * np.abs(rows).sum(0))
    assert int(torch.count_nonzero(got)) <= 2 * N


def test_embed_backward_empty():
    got = torch.full((5, 12), float("nan"), device="cuda")
    vp.embed_backward(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 12, device="cuda"), got)
    assert (got == 0).all()
    got.fill_(3.0)
    vp.embed_backward(torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 12, device="cuda"), got,
                      accumulate=True)
    assert (got == 3).all()


# ------------------------------------------------------------------ layer norm
def _ln_bounds(x, gamma, beta, mean, rstd, y, dtype):
    C = x.shape[1]
    D = C / 32 + 64
    h, t = _half(dtype)
    d_mean = (D + 2) * U * np.abs(x).mean(1)
    R = (D + 8) * U + d_mean ** 2 * rstd ** 2 / 2
    xm = np.abs(x - mean[:, None])
    by = (np.abs(gamma) * (rstd[:, None] * (d_mean[:, None] + U * xm) + xm * rstd[:, None] * (R[:, None] + 4 * U))
          + (U + h) * np.abs(y) + t)
    return by, d_mean, R * rstd


LN_SHAPES = [(1, 1), (1, 64), (3, 7), (9, 8), (5, 33), (40, 256), (577, 1001), (70, 1152), (33, 1160), (17, 2048),
             (9, 4096), (6, 5120), (5, 9216), (3, 9999), (2, 16392), (2, 70000), (2500, 72), (1300, 129),
             (1000, 1153), (301, 1279), (64, 2047), (2049, 3), (100, 8191)]


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layernorm(pair, rows, C):
    tx, ty = pair
    layout = LAYOUTS[(rows + C) % 4]
    x = _rand((rows, C), tx, 10, 2.0, 0.5)
    gamma, beta = _rand((C,), SF, 11, 0.3, 1.0), _rand((C,), SF, 12, 0.2)
    y = _place(torch.full((rows, C), float("nan"), dtype=ty), layout)
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    vp.layernorm(_place(x, layout), y, gamma.cuda(), beta.cuda(), 1e-5, mean, rstd)
    want, m, r = P.layernorm(_f64(x), _f64(gamma), _f64(beta), float(np.float32(1e-5)))
    by, bm, br = _ln_bounds(_f64(x), _f64(gamma), _f64(beta), m, r, want, ty)
    _within(mean, m, bm, "mean")
    _within(rstd, r, br + U * r, "rstd")
    _within(y, want, by, "y")
    if layout in ("padded", "odd"):
        assert (y._base[:, C:] == 77).all()
    z = torch.empty(rows, C, dtype=ty, device="cuda")
    vp.layernorm(x.cuda(), z)                                          # no weights, no statistics, dense
    want, m, r = P.layernorm(_f64(x), None, None, float(np.float32(1e-5)))
    _within(z, want, _ln_bounds(_f64(x), np.ones(C), np.zeros(C), m, r, want, ty)[0], "plain")


@pytest.mark.parametrize("C", [1, 3, 5, 6, 9, 15, 17, 31, 130])
@pytest.mark.parametrize("pair", [(BF, BF), (SF, SF), (SF, BF)])
def test_layernorm_keeps_to_its_matrices(C, pair):
    """Matrices that begin anywhere in a buffer, rows shorter than an aligned vector among
    them: what lies around them is neither used (NaN) nor written, both ways."""
    tx, ty = pair
    for rows in (1, 2, 7, 40):
        for lead in (0, 1, 3, 5):
            def within(t):
                buf = torch.full((rows * C + 32,), float("nan"), dtype=t.dtype, device="cuda")
                buf[8 + lead:8 + lead + rows * C] = t.reshape(-1).cuda()
                return buf, buf[8 + lead:8 + lead + rows * C].view(rows, C)

            def untouched(buf):
                return bool(torch.isnan(buf[:8 + lead]).all() and torch.isnan(buf[8 + lead + rows * C:]).all())

            x, d_y = _rand((rows, C), tx, rows + C), _rand((rows, C), ty, 7)
            _, xd = within(x)
            yb, y = within(torch.zeros(rows, C, dtype=ty))
            mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            vp.layernorm(xd, y, mean=mean, rstd=rstd)
            want, m, r = P.layernorm(_f64(x), None, None, float(np.float32(1e-5)))
            _within(y, want, _ln_bounds(_f64(x), np.ones(C), np.zeros(C), m, r, want, ty)[0], "y")
            assert untouched(yb)
            _, dd = within(d_y)
            db, dx = within(torch.zeros(rows, C, dtype=tx))
            dg, dbeta = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
            vp.layernorm_backward(xd, mean, rstd, dd, None, dx, dg, dbeta)
            _, wg, wb = P.layernorm_backward(_f64(x), _f64(mean), _f64(rstd), _f64(d_y))
            xhat = (_f64(x) - _f64(mean)[:, None]) * _f64(rstd)[:, None]
            _within(dg, wg, (rows + 8) * U * np.abs(_f64(d_y) * xhat).sum(0), "d_gamma")
            _within(dbeta, wb, (rows + 8) * U * np.abs(_f64(d_y)).sum(0), "d_beta")
            assert untouched(db) and not torch.isnan(dx).any()


def test_layernorm_beyond_32_bit_offsets():
    """More than 2^32 bytes, and 2^31 elements, of rows: the last ones as in a small call."""
    rows, C = 2_100_000, 1032
    x = torch.zeros(rows, C, dtype=BF, device="cuda")
    tail = _rand((3, C), BF, 15).cuda()
    x[-3:] = tail
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    vp.layernorm(x, y, mean=mean, rstd=rstd)
    small = torch.empty_like(tail)
    vp.layernorm(tail, small)
    assert torch.equal(y[-3:], small) and int(torch.count_nonzero(y[:-3])) == 0
    dx, dg = torch.empty_like(x), torch.empty(C, device="cuda")
    vp.layernorm_backward(x, mean, rstd, y, None, dx, dg)
    dx3, dg3 = torch.empty_like(tail), torch.empty(C, device="cuda")
    vp.layernorm_backward(tail, mean[-3:].clone(), rstd[-3:].clone(), small, None, dx3, dg3)
    assert torch.equal(dx[-3:], dx3) and int(torch.count_nonzero(dx[:-3])) == 0
    _within(dg, _f64(dg3), 16 * U * np.abs(_f64(dg3)))                 # three terms of one sign (d_y is xhat rounded)


def test_layernorm_offset_rows_and_leading_axes():
    """Rows whose mean is far above their spread keep their variance; a 4-D input is rows of
    its last axis; eps <= 0 is the default."""
    x = _rand((2, 3, 5, 96), SF, 13, 1.0, 1000.0).cuda()
    y, rstd = torch.empty_like(x), torch.empty(30, device="cuda")
    vp.layernorm(x, y, eps=0.0, rstd=rstd)
    flat = _f64(x).reshape(30, 96)
    want, m, r = P.layernorm(flat, eps=float(np.float32(1e-5)))
    by, _, br = _ln_bounds(flat, np.ones(96), np.zeros(96), m, r, want, SF)
    _within(y.view(30, 96), want, by)
    _within(rstd, r, br + U * r)


@pytest.mark.parametrize("C", [64, 1001, 1152, 5120, 20000])
def test_layernorm_bad_values_stay_in_their_row(C):
    x = _rand((9, C), BF, 14)
    ref = torch.empty(9, C, dtype=BF, device="cuda")
    vp.layernorm(x.cuda(), ref)
    x[2, C // 2], x[5, 0], x[7, C - 1] = float("inf"), float("nan"), float("-inf")
    got = torch.empty(9, C, dtype=BF, device="cuda")
    vp.layernorm(x.cuda(), got)
    for r in range(9):
        if r in (2, 5, 7):
            assert torch.isnan(got[r]).all()
        else:
            assert torch.equal(got[r], ref[r])
    x[:] = 3.0                                                         # no spread: zeros, not NaN
    vp.layernorm(x.cuda(), got)
    assert (got == 0).all()


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("C", [1, 7, 13, 33, 40, 257, 1001, 1152, 2000, 2600, 5120, 7168, 7618, 12000, 20000, 70000])
def test_layernorm_of_constant_rows(pair, C):
    """Every element of a row equal, to a value of 8 bits at most: every partial sum is an
    integer multiple of the value's last bit below 2^24 of them, so exact, and so are the mean,
    the differences (0) and y (beta)."""
    tx, ty = pair
    values = torch.tensor([7.0, 1000.0, 205 / 2048, -3.5, 0.0])
    x = values[:, None].expand(5, C).to(tx).contiguous()
    beta = _rand((C,), SF, 17)
    for layout in ("dense", "shifted"):
        y = _place(torch.full((5, C), float("nan"), dtype=ty), layout)
        mean, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
        vp.layernorm(_place(x, layout), y, None, beta.cuda(), 1e-5, mean, rstd)
        assert torch.equal(mean.cpu(), values)
        assert torch.equal(y.cpu(), beta.to(ty).expand(5, C))
        _within(rstd, np.full(5, float(np.float32(1e-5)) ** -0.5), 4 * U * 1e-5 ** -0.5)


@pytest.mark.parametrize("C", [7, 33, 1152, 5120, 7168, 70000])
def test_layernorm_statistics_of_infinite_rows(C):
    """The statistics go through the formula: an infinity is the mean, its square no number."""
    x = torch.zeros(3, C)
    x[0, C // 3], x[1, C - 1], x[2, 0] = float("inf"), float("-inf"), float("nan")
    y, mean, rstd = torch.zeros(3, C, device="cuda"), torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    vp.layernorm(x.cuda(), y, mean=mean, rstd=rstd)
    assert mean[:2].tolist() == [float("inf"), float("-inf")] and torch.isnan(mean[2])
    assert torch.isnan(rstd).all() and torch.isnan(y).all()


@pytest.mark.parametrize("pair", PAIRS)
@pytest.mark.parametrize("rows,C", LN_SHAPES)
def test_layernorm_backward(pair, rows, C):
    tx, ty = pair
    layout = LAYOUTS[(rows + 3 * C) % 4]
    x, d_y, gamma = _rand((rows, C), tx, 20, 2.0, 0.5), _rand((rows, C), ty, 21), _rand((C,), SF, 22, 0.3, 1.0)
    _, mean, rstd = P.layernorm(_f64(x))
    mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
    x64, dy64, g64, m64, r64 = (_f64(t) for t in (x, d_y, gamma, mean, rstd))
    want_dx, want_dg, want_db = P.layernorm_backward(x64, m64, r64, dy64, g64)
    xhat, g = (x64 - m64[:, None]) * r64[:, None], dy64 * g64
    D, (h, t) = C / 32 + 64, _half(tx)
    mg, mgx = np.abs(g).mean(1, keepdims=True), np.abs(g * xhat).mean(1, keepdims=True)
    # xhat's two roundings also reach the mean of g * xhat: in (D + 8)
    bdx = (r64[:, None] * (3 * U * np.abs(g) + (D + 3) * U * mg + np.abs(xhat) * (D + 8) * U * mgx
                           + 6 * U * np.abs(xhat) * np.abs((g * xhat).mean(1, keepdims=True)))
           + (4 * U + h) * np.abs(want_dx) + t)
    bdg, bdb = (rows + 8) * U * np.abs(dy64 * xhat).sum(0), (rows + 8) * U * np.abs(dy64).sum(0)
    xd, dd = _place(x, layout), _place(d_y, layout)
    dx = _place(torch.full((rows, C), float("nan"), dtype=tx), layout)
    dg, db = (torch.full((C,), float("nan"), device="cuda") for _ in range(2))
    args = (xd, mean.cuda(), rstd.cuda(), dd)
    vp.layernorm_backward(*args, gamma.cuda(), dx, dg, db)
    _within(dx, want_dx, bdx, "d_x")
    _within(dg, want_dg, bdg, "d_gamma")
    _within(db, want_db, bdb, "d_beta")
    if layout in ("padded", "odd"):
        assert (dx._base[:, C:] == 77).all()
    # each output alone gives the same values; without gamma it is one
    dx1 = _place(torch.full((rows, C), float("nan"), dtype=tx), layout)
    vp.layernorm_backward(*args, gamma.cuda(), d_x=dx1)
    _within(dx1, want_dx, bdx, "d_x alone")
    dg1, db1 = torch.empty_like(dg), torch.empty_like(db)
    vp.layernorm_backward(*args, gamma.cuda(), d_gamma=dg1)
    vp.layernorm_backward(*args, d_beta=db1)
    _within(dg1, want_dg, bdg, "d_gamma alone")
    _within(db1, want_db, bdb, "d_beta alone")
    dx2, dg2 = _place(torch.full((rows, C), float("nan"), dtype=tx), layout), torch.empty_like(dg)
    vp.layernorm_backward(*args, gamma.cuda(), dx2, dg2, db1)
    assert torch.equal(dg2, dg) and torch.equal(dx2, dx)               # a fixed order for one layout


@pytest.mark.parametrize("C", [64, 1001, 5120])
def test_layernorm_backward_of_rows_without_spread(C):
    """Zero variance under a tiny eps: rstd 1e20, whose square no fp32 holds, meets xhat = 0."""
    x, d_y = torch.full((3, C), 2.0, device="cuda"), torch.ones(3, C, device="cuda")
    mean, rstd = torch.full((3,), 2.0, device="cuda"), torch.full((3,), 1e20, device="cuda")
    d_x, dg, db = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    vp.layernorm_backward(x, mean, rstd, d_y, None, d_x, dg, db)
    # g - mean(g): a sum of C ones is exact, its mean off by at most one rounding of 1/C
    assert (d_x.abs() <= 1e20 * 2.0 ** -23).all() and (dg == 0).all() and (db == 3).all()


def test_layernorm_backward_empty():
    dg, db = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
    e = torch.empty(0, 40, dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    vp.layernorm_backward(e, s, s, e, None, torch.empty_like(e), dg, db)
    assert (dg == 0).all() and (db == 0).all()


# ------------------------------------------------------------------ clipping
def _clip_case(sizes, dtypes, seed, scale=1.0, shift=0):
    ts = []
    for i, n in enumerate(sizes):
        t = _rand((n + shift,), dtypes[i % len(dtypes)], seed + i, scale)
        ts.append(t)
    return ts


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [20_000] * 13, [262_144], [262_141, 3], [262_145], [3] * 16, [3] * 17, [8192, 8193, 1, 7], [100_003], [64, 1 << 20, 33], [9] * 1000,
                                   [16384, 0, 256, 32768, 128, 64, 64]])
@pytest.mark.parametrize("dtypes", [[SF], [BF], [HF], [SF, BF, HF]])
@pytest.mark.parametrize("shift", [0, 1])
def test_clip(sizes, dtypes, shift):
    ts = _clip_case(sizes, dtypes, 30, 1.0, shift)
    dev = [t.cuda()[shift:] for t in ts]
    g64 = [_f64(t) for t in dev]
    for max_norm in (0.5, 0.0, 1e6):
        want_norm, want = P.clip_grads(g64, max_norm)
        norm = torch.full((1,), float("nan"), device="cuda")
        out = [torch.full_like(t, float("nan")) for t in dev]
        vp.clip_grads(dev, max_norm, norm, out)
        for t, w in zip(out, want):
            h, sub = _half(t.dtype)
            _within(t, w, np.abs(w) * (h + 11 * U) + sub)
        _within(norm, np.array([want_norm]), 8 * U * want_norm)
        only = torch.empty(1, device="cuda")
        vp.grad_norm(dev, only)
        assert torch.equal(only, norm)
        inplace = [t.clone() for t in dev]
        vp.clip_grads(inplace, max_norm)
        for a, b in zip(inplace, out):
            assert torch.equal(a, b)
    for t, g in zip(dev, g64):
        assert (_f64(t) == g).all()                                     # inputs stay


def test_clip_beyond_32_bit_offsets():
    t = torch.zeros((1 << 31) + 77, dtype=BF, device="cuda")
    t[-1], t[0] = 4.0, 3.0
    norm = torch.empty(1, device="cuda")
    vp.clip_grads([t], 1.0, norm)
    assert float(norm) == 5.0 and int(torch.count_nonzero(t)) == 2
    want = P.clip_grads([np.array([3.0, 4.0])], 1.0)[1][0]
    _within(torch.stack([t[0], t[-1]]), want, want * (2.0 ** -8 + 11 * U))


def test_clip_extreme_values():
    # squares above fp32's largest and below its smallest value
    for scale in (1e25, 1e-30, 1e-38):
        ts = [_rand((5000,), SF, 40, scale).cuda(), _rand((77,), SF, 41, scale).cuda()]
        norm = torch.empty(1, device="cuda")
        out = [torch.empty_like(t) for t in ts]
        vp.clip_grads(ts, scale, norm, out)
        want_norm, want = P.clip_grads([_f64(t) for t in ts], scale)
        _within(norm, np.array([want_norm]), 8 * U * want_norm + 2.0 ** -150)
        for t, w in zip(out, want):
            _within(t, w, np.abs(w) * 12 * U + 2.0 ** -150)
    # a coefficient below fp32's normal range
    ts = [torch.full((9,), 3e38, device="cuda")]
    out = [torch.empty_like(ts[0])]
    vp.clip_grads(ts, 1e-3, None, out)
    want = P.clip_grads([_f64(ts[0])], 1e-3)[1][0]
    _within(out[0], want, np.abs(want) * 12 * U)


def test_clip_infinities_and_nan():
    for bad in (float("inf"), float("-inf"), float("nan")):
        t = torch.ones(20_000, device="cuda")
        t[12_345] = bad
        u = torch.ones(5, dtype=BF, device="cuda")
        norm = torch.empty(1, device="cuda")
        want_norm, want = P.clip_grads([_f64(t), _f64(u)], 1.0)
        vp.clip_grads([t, u], 1.0, norm)
        np.testing.assert_array_equal(_f64(norm), [want_norm])
        np.testing.assert_array_equal(_f64(t), want[0])
        np.testing.assert_array_equal(_f64(u), want[1])


def test_clip_takes_the_dict_backward_fills():
    grads = {"W1": _rand((64, 32), SF, 50).cuda(), "b1": None, "W_mid": [_rand((8, 8), SF, 51).cuda(), None],
             "b2": _rand((7,), SF, 52).cuda()}
    flat = [_f64(grads["W1"]), _f64(grads["W_mid"][0]), _f64(grads["b2"])]
    want_norm, want = P.clip_grads(flat, 1.0)
    norm = torch.empty(1, device="cuda")
    vp.clip_grads(grads, 1.0, norm)
    _within(norm, np.array([want_norm]), 8 * U * want_norm)
    for t, w in zip((grads["W1"], grads["W_mid"][0], grads["b2"]), want):
        _within(t, w, 12 * U * np.abs(w))


# ------------------------------------------------------------------ streams, graphs, together
def _step(ids, table, x, gamma, beta, d_out, bufs, stream=None):
    """The operators in the order of a training step: text rows, layer norm of the features,
    its gradients, the table's gradient, clipping of all of them."""
    vp.embed(ids, table, bufs["seq"], scale=8.0, image_token_id=TOKEN, stream=stream)
    vp.layernorm(x, bufs["y"], gamma, beta, 1e-5, bufs["mean"], bufs["rstd"], stream=stream)
    vp.layernorm_backward(x, bufs["mean"], bufs["rstd"], bufs["y"], gamma, bufs["dx"], bufs["dg"], bufs["db"],
                          stream=stream)
    vp.embed_backward(ids, d_out, bufs["dt"], scale=8.0, image_token_id=TOKEN, stream=stream)
    vp.clip_grads([bufs["dt"], bufs["dg"], bufs["db"]], 1.0, bufs["norm"], stream=stream)


def _step_inputs(seed, n=3000, N=64, vocab=500, rows=900, C=96):
    ids = _ids("mixed", n, vocab, seed).cuda()
    table, x = _rand((vocab, N), BF, seed + 1).cuda(), _rand((rows, C), BF, seed + 2).cuda()
    gamma, beta = _rand((C,), SF, seed + 3, 0.1, 1.0).cuda(), _rand((C,), SF, seed + 4).cuda()
    return ids, table, x, gamma, beta, _rand((n, N), BF, seed + 5).cuda()


def _step_bufs(n=3000, N=64, vocab=500, rows=900, C=96):
    e = lambda *s, dtype=SF: torch.zeros(*s, dtype=dtype, device="cuda")      # noqa: E731
    return {"seq": e(n, N, dtype=BF), "y": e(rows, C, dtype=BF), "mean": e(rows), "rstd": e(rows),
            "dx": e(rows, C, dtype=BF), "dg": e(C), "db": e(C), "dt": e(vocab, N), "norm": e(1)}


def test_step_on_streams_and_in_graphs():
    ins = [_step_inputs(100), _step_inputs(200)]
    want = []
    for i in ins:
        b = _step_bufs()
        _step(*i, b)
        want.append({k: v.clone() for k, v in b.items()})
    torch.cuda.synchronize()
    # two streams at once, the workspaces taken for each call on its own stream
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = [_step_bufs(), _step_bufs()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, b, s in zip(ins, bufs, streams):
            _step(*i, b, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert all(torch.equal(b[k], w[k]) for k in w)
    # a raw stream address, and the default stream by its address
    for raw in (streams[0].cuda_stream, 0):
        b = _step_bufs()
        torch.cuda.synchronize()
        _step(*ins[1], b, stream=raw)
        torch.cuda.synchronize()
        assert all(torch.equal(b[k], want[1][k]) for k in want[1])
    # two captured graphs replayed at the same time, new inputs copied in between
    graphs, bufs = [], [_step_bufs(), _step_bufs()]
    held = [[t.clone() for t in i] for i in ins]
    for i, b in zip(held, bufs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(*i, b)
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for k, h in enumerate(held):
            for dst, src in zip(h, ins[order[k]]):
                dst.copy_(src)
        torch.cuda.synchronize()
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for k, b in enumerate(bufs):
            assert all(torch.equal(b[q], want[order[k]][q]) for q in b)


def test_step_from_several_host_threads():
    """Calls of four threads at once, each on its own stream: the library's tables of the
    device are shared between them."""
    import threading

    ins = [_step_inputs(400 + k) for k in range(4)]
    bufs, streams = [_step_bufs() for _ in ins], [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(ins))

    def run(i, b, s):
        try:
            start.wait()
            for _ in range(30):
                _step(*i, b, stream=s)
        except Exception as e:                                         # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=a) for a in zip(ins, bufs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i, b in zip(ins, bufs):
        want = _step_bufs()
        _step(*i, want)
        assert all(torch.equal(b[k], want[k]) for k in want)


def test_given_workspaces():
    ids, table, x, gamma, beta, d_out = _step_inputs(300)
    dt, dt2 = torch.empty(500, 64, device="cuda"), torch.empty(500, 64, device="cuda")
    w = torch.full((vp.embed_backward_workspace(3000, 64),), 255, dtype=torch.uint8, device="cuda")
    vp.embed_backward(ids, d_out, dt, image_token_id=TOKEN, workspace=w)
    vp.embed_backward(ids, d_out, dt2, image_token_id=TOKEN)
    assert torch.equal(dt, dt2)
    w = torch.full((vp.clip_grads_workspace(1),), 255, dtype=torch.uint8, device="cuda")
    norm, norm2 = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    vp.grad_norm([dt], norm, workspace=w)
    vp.grad_norm([dt], norm2)
    assert torch.equal(norm, norm2)
    mean, rstd, dg, dg2 = (torch.empty(k, device="cuda") for k in (900, 900, 96, 96))
    vp.layernorm(x, torch.empty_like(x), mean=mean, rstd=rstd)
    w = torch.full((vp.layernorm_backward_workspace(900, 96),), 255, dtype=torch.uint8, device="cuda")
    vp.layernorm_backward(x, mean, rstd, x, d_gamma=dg, workspace=w)
    vp.layernorm_backward(x, mean, rstd, x, d_gamma=dg2)
    assert torch.equal(dg, dg2)


def test_training_step_around_the_projector():
    """Text rows by vp.embed, image rows by the projector, its gradients and the table's from
    one loss gradient, all clipped together; the projector's own results do not change."""
    import workloads as W
    from gpu_harness import DeviceInputs, check, dev_bf16, make_case, make_projector

    case = make_case(W.WORKLOADS["tiny"])
    wl = case.wl
    proj, dev = make_projector(case), DeviceInputs(case)
    out = torch.empty_like(dev.prefill)
    vp.embed(dev.ids, dev_bf16(W.embed_table(wl)), out, image_token_id=W.IMAGE_TOKEN_ID)
    proj.forward(dev.feats, case.hw, None, dev.ids, W.IMAGE_TOKEN_ID, out)
    assert proj.status() == vp.OK
    check(case, out, dev)
    d_out = dev_bf16(W.grad_out(wl, len(case.ids)))
    shapes = {"W1": (wl.N1, wl.K1), "b1": (wl.N1,), "W2": (wl.N2, wl.N1), "b2": (wl.N2,), "gamma": (wl.C,),
              "beta": (wl.C,)}
    grads = {k: torch.empty(s, device="cuda") for k, s in shapes.items()}
    proj.backward(dev.feats, case.hw, None, dev.ids, W.IMAGE_TOKEN_ID, d_out, grads)
    d_table = torch.empty(W.TEXT_VOCAB, wl.N2, device="cuda")
    vp.embed_backward(dev.ids, d_out, d_table, image_token_id=W.IMAGE_TOKEN_ID)
    want_t, mag = P.embed_backward(case.ids, _f64(d_out), W.TEXT_VOCAB, 1.0, W.IMAGE_TOKEN_ID)
    _within(d_table, want_t, 40 * U * mag)
    every = dict(grads, table=d_table)
    before = [_f64(t) for t in every.values()]
    norm = torch.empty(1, device="cuda")
    vp.clip_grads(every, 1.0, norm)
    want_norm, want = P.clip_grads(before, 1.0)
    _within(norm, np.array([want_norm]), 8 * U * want_norm)
    for t, w in zip(every.values(), want):
        _within(t, w, 12 * U * np.abs(w))


# ------------------------------------------------------------------ empty tables, ids without placeholders
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_ids_of_an_empty_table_are_latched(n):
    """No id lies inside a table of no rows: lookup and table gradient both say so, by either
    way of summing."""
    ids = torch.arange(n).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.ones(n, 8, device="cuda")
    vp.embed(ids, torch.empty(0, 8, device="cuda"), out, status=status)
    assert int(status) == vp.ERR_INVALID_ARG and int(torch.count_nonzero(out)) == 0
    status.zero_()
    vp.embed_backward(ids, out, torch.empty(0, 8, device="cuda"), status=status)
    assert int(status) == vp.ERR_INVALID_ARG
    status.zero_()
    ids.fill_(TOKEN)
    vp.embed_backward(ids, out, torch.empty(0, 8, device="cuda"), image_token_id=TOKEN, status=status)
    assert int(status) == vp.OK                                        # placeholders only


@pytest.mark.parametrize("n", [6, 3000])
def test_lowest_id_is_outside_the_table(n):
    """Without placeholders an id of the lowest int64 value is a bad id like any other."""
    ids = torch.zeros(n, dtype=torch.int64)
    ids[1] = vp.NO_TOKEN
    table, out = torch.full((3, 8), 2.0, device="cuda"), torch.ones(n, 8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vp.embed(ids.cuda(), table, out, status=status)
    assert int(status) == vp.ERR_INVALID_ARG and (out[1] == 0).all() and (out[2] == 2).all()
    status.zero_()
    d_table = torch.empty(3, 8, device="cuda")
    vp.embed_backward(ids.cuda(), torch.ones(n, 8, device="cuda"), d_table, status=status)
    assert int(status) == vp.ERR_INVALID_ARG and (d_table[0] == n - 1).all() and (d_table[1:] == 0).all()
