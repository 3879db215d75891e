"""The operators at the ends of the model against plain 64-bit implementations.

Tolerances are bounds per element, from the roundings that the formulas and the
kernels' order of sums allow (u = 2^-24, half a step of fp32; h = half a step of
the type), not measured figures.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu



@pytest.fixture(scope="module", autouse=True)
def leave_nothing():
    """Tensors that closures and caught exceptions still hold in cycles are freed here,
    not at some later moment in a test that watches the allocator."""
    yield
    import gc
    gc.collect()
    torch.cuda.empty_cache()


BF, FP = torch.bfloat16, torch.float32
U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def check(got, want, tol, what=""):
    """|got - want| <= tol for every element (and finite where want is)."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((d / tol.clamp(min=1e-300)).max()))


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,v,d,idt", [(1, 1, 8, torch.int64), (3, 7, 8, torch.int32), (67, 515, 64, torch.int64),
                                       (1025, 33, 2056, torch.int32), (4099, 50021, 256, torch.int64)])
def test_embed(n, v, d, idt, dtype):
    from recurrent_memory_transformer_diag_b200 import embed
    g = gen(n + v)
    table = randn(g, v, d).to(dtype)
    ids = torch.randint(-2, v + 2, (n,), generator=g, device="cuda").to(idt)
    if n > 1:
        ids[0] = -1
    scale = 1.7
    out = torch.full((n, d), float("nan"), dtype=dtype, device="cuda")
    embed(ids, table, out, scale=scale)
    ok = (ids >= 0) & (ids < v)
    want = torch.where(ok[:, None], table.double()[ids.long().clamp(0, v - 1)] * scale, 0.0)
    # the scale as fp32, the product in fp32, then the type
    check(out, want, want.abs() * (half(dtype) + 2.5 * U) + 1e-38)
    embed(ids, table, out)   # scale 1: a copy
    assert torch.equal(out, torch.where(ok[:, None], table[ids.long().clamp(0, v - 1)], torch.zeros_like(out)))


def grad_reference(ids, d_out, v, scale, base):
    ok = (ids >= 0) & (ids < v)
    i, x = ids[ok].long(), d_out[ok].double()
    z = torch.zeros(v, d_out.shape[1], dtype=torch.float64, device="cuda")
    s, a = z.index_add(0, i, x) * scale, z.index_add(0, i, x.abs()) * abs(scale)
    count = torch.bincount(i, minlength=v).double()[:, None]
    return s + base, a, count


EMBED_GRAD = [
    # n, v, d, how the ids fall
    (1, 1, 8, "uniform"), (1, 300, 64, "uniform"), (67, 515, 64, "uniform"),
    (128, 100, 72, "skewed"),              # most tokens of the one-launch form
    (128, 40, 64, "one"),
    (129, 100, 72, "skewed"),              # fewest of the sorted one
    (2048, 1000, 72, "skewed"), (2048, 40, 64, "one"), (2049, 1000, 72, "skewed"),
    (2049, 1, 8, "uniform"),               # one row takes everything
    (5000, 511, 64, "uniform"), (5000, 512, 64, "uniform"), (5000, 262145, 8, "uniform"),   # 1, 2, 3 passes
    (20011, 3001, 256, "skewed"), (9000, 100, 2048, "one"), (6400, 100, 64, "blocks"),
    (4097, 77, 2056, "skewed"),            # columns in two blocks
    (3000, 50, 16, "none"), (8192, 300, 64, "skewed"), (8193, 300, 64, "skewed"), (12000, 511, 64, "uniform"),
    (12000, 512, 64, "uniform"), (12000, 262145, 8, "uniform"), (9000, 5, 64, "none"),
]


def make_ids(g, n, v, how):
    if how == "uniform":
        return torch.randint(0, v, (n,), generator=g, device="cuda")
    if how == "one":
        return torch.full((n,), v // 2, device="cuda", dtype=torch.int64)
    if how == "none":
        return torch.full((n,), -1, device="cuda", dtype=torch.int64)
    if how == "blocks":   # runs that end exactly at multiples of 64
        return (torch.arange(n, device="cuda") // 64) % v
    ids = (v * torch.rand(n, generator=g, device="cuda") ** 4).long().clamp_(max=v - 1)
    ids[torch.rand(n, generator=g, device="cuda") < 0.1] = -100
    return ids


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,v,d,how", EMBED_GRAD)
def test_embed_grad(n, v, d, how, dtype, accumulate):
    from recurrent_memory_transformer_diag_b200 import embed_grad
    g = gen(n + v + d)
    ids = make_ids(g, n, v, how)
    d_out = randn(g, n, d).to(dtype)
    base = randn(g, v, d).to(dtype)
    scale = 0.75
    out = base.clone() if accumulate else torch.full_like(base, float("nan"))
    embed_grad(ids, d_out, out, scale=scale, accumulate=accumulate)
    want, absum, count = grad_reference(ids, d_out, v, scale, base.double() if accumulate else 0.0)
    # a sum of k terms in any fixed order, the scale, the base, the type
    check(out, want, absum * (count + 3) * U + want.abs() * (half(dtype) + U) + 1e-38)
    if accumulate:   # rows that no token names keep their bits
        assert torch.equal(out[count[:, 0] == 0], base[count[:, 0] == 0])
    again = base.clone() if accumulate else torch.empty_like(base)
    embed_grad(ids.to(torch.int32), d_out, again, scale=scale, accumulate=accumulate)
    assert torch.equal(again, out)   # no order left to chance; int32 ids alike


def test_embed_grad_is_the_gradient_of_embed():
    """<d_out, embed(table + e) - embed(table)> = <d_table, e> for exact values
    (small integers: every sum below 2^24 is exact)."""
    from recurrent_memory_transformer_diag_b200 import embed, embed_grad
    g = gen(5)
    n, v, d = 3001, 97, 40
    table = torch.randint(-8, 9, (v, d), generator=g, device="cuda").float()
    e = torch.randint(-3, 4, (v, d), generator=g, device="cuda").float()
    d_out = torch.randint(-4, 5, (n, d), generator=g, device="cuda").float()
    ids = torch.randint(-1, v, (n,), generator=g, device="cuda")
    a, b = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda")
    embed(ids, table, a, scale=2.0)
    embed(ids, table + e, b, scale=2.0)
    d_table = torch.empty(v, d, device="cuda")
    embed_grad(ids, d_out, d_table, scale=2.0)
    assert float((d_out.double() * (b - a).double()).sum()) == float((d_table.double() * e.double()).sum())


def test_embed_masked_values():
    """NaN and infinities of padding rows do not reach the table's gradient."""
    from recurrent_memory_transformer_diag_b200 import embed_grad
    for n in (100, 4000):
        ids = torch.arange(n, device="cuda") % 13
        ids[::3] = -1
        d_out = torch.ones(n, 16, device="cuda")
        d_out[::3] = float("nan")
        d_out[0] = float("inf")
        out = torch.empty(20, 16, device="cuda")
        embed_grad(ids, d_out, out)
        want = torch.bincount(ids[ids >= 0], minlength=20).double()[:, None].expand(20, 16)
        assert torch.equal(out.double(), want)


# ------------------------------------------------------------------ norm
NORM = [(1, 8), (7, 64), (33, 256), (5, 264), (9, 1000), (65, 2048), (11, 2056), (3, 4096), (4, 8192), (2, 16384),
        (3000, 512), (700, 2048)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,d", NORM)
def test_rms_norm_and_gradient(n, d, dtype):
    from recurrent_memory_transformer_diag_b200 import rms_norm, rms_norm_grad
    g = gen(n + d)
    x = (randn(g, n, d) * torch.exp(2 * randn(g, n, 1))).to(dtype)
    gain = (1 + 0.3 * randn(g, d)).to(dtype)
    dy = randn(g, n, d).to(dtype)
    eps = 1e-5
    y, rstd = torch.empty_like(x), torch.empty(n, device="cuda")
    rms_norm(x, gain, y, rstd, eps)
    X, G, D = x.double(), gain.double(), dy.double()
    R = ((X * X).mean(1, keepdim=True) + eps) ** -0.5
    # a lane adds at most d / 32 squares, then 5 + 8 sums; half of that reaches the root, plus rsqrt's 2 ulp
    er = (d / 32 + 16) * U / 2 + 6 * U
    check(rstd[:, None], R, R * er)
    Y = X * R * G
    check(y, Y, Y.abs() * (er + 3 * U + half(dtype)) + 1e-38)
    dx, d_gain = torch.full_like(x, float("nan")), torch.full_like(gain, float("nan"))
    rms_norm_grad(x, gain, rstd, dy, dx, d_gain)
    M = (D * G * X).mean(1, keepdim=True)
    Ma = (D * G * X).abs().mean(1, keepdim=True)
    want = R * (D * G - X * R * R * M)
    mag = R * ((D * G).abs() + X.abs() * R * R * Ma)
    check(dx, want, mag * (3 * er + (d / 32 + 16) * U + 8 * U) + want.abs() * half(dtype) + 1e-38)
    wg = (D * X * R).sum(0)
    mag = (D * X * R).abs().sum(0)
    # a block's warp adds its rows, 8 warps, at most 10 partial sums in a group, 32 groups
    check(d_gain, wg, mag * (er + (n / 8 + 8 + 10 + 32 + 3) * U) + wg.abs() * half(dtype) + 1e-38)
    # in place
    y2, dx2 = x.clone(), dy.clone()
    rms_norm(y2, gain, y2, None, eps)
    assert torch.equal(y2, y)
    rms_norm_grad(x, gain, rstd, dx2, dx2, torch.empty_like(gain))
    assert torch.equal(dx2, dx)


def test_rms_norm_zero_row():
    from recurrent_memory_transformer_diag_b200 import rms_norm, rms_norm_grad
    x = torch.zeros(3, 64, device="cuda")
    x[1] = 1.0
    gain = torch.ones(64, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(3, device="cuda")
    rms_norm(x, gain, y, rstd, 1e-6)
    assert torch.equal(y[0], x[0]) and torch.allclose(rstd[0], torch.tensor(1e3, device="cuda"))
    dx, dg = torch.empty_like(x), torch.empty_like(gain)
    rms_norm_grad(x, gain, rstd, torch.ones_like(x), dx, dg)
    assert torch.isfinite(dx).all() and torch.allclose(dx[0], torch.full((64,), 1e3, device="cuda"))


# ------------------------------------------------------------------ vocabulary loss
def loss_reference(hidden, head, targets, scale):
    """logits, lse, loss, sum |h w| (64 bits), and which rows count."""
    H, W = hidden.double(), head.double()
    ok = (targets >= 0) & (targets < head.shape[0])
    H = torch.where(ok[:, None], H, 0.0)
    L = H @ W.t() * scale
    lse = torch.logsumexp(L, 1)
    t = targets.long().clamp(0, head.shape[0] - 1)[:, None]
    loss = torch.where(ok, lse - L.gather(1, t)[:, 0], 0.0)
    A = (H.abs() @ W.abs().t()).max(1).values * abs(scale)
    return L, torch.where(ok, lse, 0.0), loss, A, ok


def logit_error(A, d, planes):
    """A logit's error: a chunk of at most 32 instructions (K = 512), each truncated (2 u) once
    in the instruction's own sum and once in the accumulator, chunks (of 128 at least) added
    to nearest; fp32 operands: chunks of a k-block's six products (24 instructions), and three
    terms of 24 bits less what the dropped products hold.  Plain multiply-adds (d / 128 a lane,
    5 sums) stay below that."""
    chunks = math.ceil(d / 64) / (1 if planes == 3 else 2)
    return A * ((64 * 2 + chunks) * U + (8 * U if planes == 3 else 0))


def loss_inputs(seed, n, v, d, dtype, idt=torch.int64, ignored=0.2):
    g = gen(seed)
    head = (randn(g, v, d) / math.sqrt(d)).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    hidden = (randn(g, n, d) + 8 * torch.rand(n, 1, generator=g, device="cuda") * head[t].float()).to(dtype)
    t[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    w = (0.5 + torch.rand(n, generator=g, device="cuda")) / n
    return hidden, head, t.to(idt), w


def run_loss(hidden, head, t, w, scale=1.0, **kw):
    from recurrent_memory_transformer_diag_b200 import token_loss, token_loss_grad
    n = hidden.shape[0]
    loss = torch.full((n,), float("nan"), device="cuda")
    lse = torch.full((n,), float("nan"), device="cuda")
    token_loss(hidden, head, t, loss, lse, scale=scale)
    dh, dw = torch.full_like(hidden, float("nan")), torch.full_like(head, float("nan"))
    token_loss_grad(hidden, head, t, lse, w, dh, dw, scale=scale, **kw)
    return loss, lse, dh, dw


def check_loss(hidden, head, t, w, scale, got):
    loss, lse, dh, dw = got
    dtype, d, v = hidden.dtype, hidden.shape[1], head.shape[0]
    planes = 3 if dtype == FP else 1
    L, rl, rloss, A, ok = loss_reference(hidden, head, t, scale)
    el = logit_error(A, d, planes) + L.abs().max(1).values * U   # and the product with the scale
    # exponentials and their sum: 2^-22 each, the sum over 128 columns and the tiles; log, the last sums
    es = (16 + 64 + v / 256) * U
    check(loss, rloss, 2 * el + es + 4 * U * (rl.abs() + rloss.abs() + 1) + 1e-30, "loss")
    check(lse, rl, el + es + 4 * U * (rl.abs() + 1) + 1e-30, "lse")
    assert (loss[~ok] == 0).all() and (lse[~ok] == 0).all()
    g = torch.where(ok, w.double(), 0.0)[:, None]
    P = torch.exp(L - rl[:, None]) * g
    at = t.long().clamp(0, v - 1)[:, None]
    onehot = torch.zeros_like(P).scatter_add_(1, at, g)
    H, W = torch.where(ok[:, None], hidden.double(), 0.0), head.double()
    # P: the logits' and the lse's error, the exponent's product, ex2, the division of the weight,
    # the subtraction; then three terms or one
    gap = (L - rl[:, None]).abs()
    ep = P.abs() * (2 * el + es + 4 * U * (rl.abs() + 1))[:, None] + P.abs() * (gap * 3 + 8) * U + onehot.abs() * 4 * U
    Q = P - onehot
    ep = ep + Q.abs() * (2 * U if planes == 3 else half(BF))
    # an exponential below 2^-126, the smallest normal fp32 number, is flushed to zero: exp(l - lse)
    # is then off by up to 2^-126 itself, P by that times its weight
    ep = ep + g.abs() * 2.0 ** -126
    # products: fp32 operands in chunks of 24 instructions (2 u twice each), added to nearest, and
    # their splits; bf16 over the whole contraction
    def chain(k):
        if planes == 3:
            return (96 + math.ceil(k / 64) + 16) * U
        return (k / 16 + 2) * 4 * U
    want = Q @ W * scale
    mag = (Q.abs() @ W.abs()) * abs(scale)
    check(dh, want, (ep @ W.abs()) * abs(scale) + mag * (chain(v) + 24 * U) + want.abs() * half(dtype) + 1e-38, "d_hidden")
    assert (dh[~ok] == 0).all()
    want = Q.t() @ H * scale
    mag = (Q.abs().t() @ H.abs()) * abs(scale)
    check(dw, want, (ep.t() @ H.abs()) * abs(scale) + mag * (chain(len(t)) + 8 * U) + want.abs() * half(dtype) + 1e-38,
          "d_head")


LOSS = [
    # n, v, d
    (1, 1, 8), (1, 300, 64), (2, 255, 72), (3, 256, 64), (5, 257, 136), (127, 512, 256), (128, 1000, 64),
    (129, 1023, 328), (255, 1025, 64), (257, 777, 512), (300, 5003, 128), (64, 33000, 64), (1030, 259, 2048),
    (4, 20000, 72), (16, 700, 200), (17, 515, 64), (65, 300, 64), (16, 300, 3208), (2000, 300, 64), (1500, 1025, 136), (130, 2500, 136), (128, 700, 384),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,v,d", LOSS)
def test_token_loss_and_gradient(n, v, d, dtype):
    scale = 1.0 if n % 2 else 0.37
    hidden, head, t, w = loss_inputs(n + v + d, n, v, d, dtype, torch.int32 if n % 2 else torch.int64,
                                     0.0 if n < 4 else 0.2)
    got = run_loss(hidden, head, t, w, scale)
    check_loss(hidden, head, t, w, scale, got)
    for a, b in zip(got, run_loss(hidden, head, t, w, scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n,v,d,dtype", [
    (8200, 300, 64, BF),       # two passes over the rows
    (8192, 17000, 64, BF),     # two pieces of the vocabulary in the gradient, the second ragged
    (4100, 11003, 64, FP),     # the same for fp32 operands
    (20011, 515, 32, BF),      # rows counted before they are ordered
    (17000, 257, 24, FP),
])
def test_token_loss_in_pieces(n, v, d, dtype):
    hidden, head, t, w = loss_inputs(n, n, v, d, dtype)
    check_loss(hidden, head, t, w, 1.0, run_loss(hidden, head, t, w))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_token_loss_masked_rows(dtype):
    """Rows without a target hold NaN and infinities, also in lse and d_loss: they
    change nothing; targets at and past the vocabulary's end are no targets."""
    n, v, d = 301, 600, 64
    hidden, head, t, w = loss_inputs(9, n, v, d, dtype)
    t[:4] = torch.tensor([-1, v, v + 5, -(1 << 40)], device="cuda")
    t[-1] = -100
    off = (t < 0) | (t >= v)
    clean = run_loss(hidden, head, t, w)
    dirty, wd = hidden.clone(), w.clone()
    dirty[off] = float("nan")
    dirty[off.nonzero()[::2, 0]] = float("inf")
    wd[off] = float("nan")
    for a, b in zip(clean, run_loss(dirty, head, t, wd)):
        assert torch.equal(a, b)
    check_loss(hidden, head, t, w, 1.0, clean)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_token_loss_no_targets_and_zero_weights(dtype):
    n, v, d = 70, 300, 64
    hidden, head, t, w = loss_inputs(3, n, v, d, dtype)
    loss, lse, dh, dw = run_loss(hidden, head, torch.full_like(t, -1), w)
    for x in (loss, lse, dh, dw):
        assert (x == 0).all()
    loss, lse, dh, dw = run_loss(hidden, head, t, torch.zeros_like(w))
    assert (loss[t >= 0] > 0).all() and (dh == 0).all() and (dw == 0).all()


def test_token_loss_large_logits():
    """Logits far beyond exp's range, a sure and a hopeless prediction."""
    n, v, d = 64, 512, 64
    hidden, head, t, w = loss_inputs(1, n, v, d, BF, ignored=0.0)
    hidden = (hidden.float() * 300).to(BF)
    got = run_loss(hidden, head, t, w)
    assert torch.isfinite(got[0]).all() and float(got[1].max()) > 1000
    check_loss(hidden, head, t, w, 1.0, got)


def test_token_loss_not_a_number():
    """A NaN in a row with a target shows in that row's loss and gradient only."""
    n, v, d = 40, 300, 64
    hidden, head, t, w = loss_inputs(2, n, v, d, FP, ignored=0.0)
    clean = run_loss(hidden, head, t, w)
    bad = hidden.clone()
    bad[7, 3] = float("nan")
    loss, lse, dh, dw = run_loss(bad, head, t, w)
    rest = torch.arange(n, device="cuda") != 7
    assert torch.isnan(loss[7]) and torch.equal(loss[rest], clean[0][rest])
    assert torch.isnan(dh[7]).all() and torch.equal(dh[rest], clean[2][rest])
    assert torch.isnan(dw).any()


def test_token_loss_range_of_fp32():
    """Numbers above bf16's largest and tiny ones (all three terms still normal) keep their value."""
    n, v, d = 33, 300, 64
    hidden, head, t, w = loss_inputs(5, n, v, d, FP, ignored=0.0)
    hidden[0], head[:, 0] = 0.0, 0.0
    hidden[0, 0] = 3.4e38
    head[7, 0] = 1e-30
    head[8, 0] = -2e-30
    got = run_loss(hidden, head, t, w)
    check_loss(hidden, head, t, w, 1.0, got)


def test_token_loss_weight_range():
    """Weights of very different and very small size, a negative one, a single one."""
    n, v, d = 130, 400, 64
    hidden, head, t, w = loss_inputs(4, n, v, d, FP, ignored=0.0)
    w = w * torch.logspace(-3, 3, n, device="cuda")
    w[5] = -w[5]
    check_loss(hidden, head, t, w, 1.0, run_loss(hidden, head, t, w))
    w = w * 1e-30
    got = run_loss(hidden, head, t, w)
    check_loss(hidden, head, t, w, 1.0, got)
    one = torch.zeros(n, device="cuda")
    one[11] = 1.0
    check_loss(hidden, head, t, one, 1.0, run_loss(hidden, head, t, one))


@pytest.mark.parametrize("n", [30, 200])
def test_token_loss_bad_weights(n):
    """An infinite and a NaN weight show in their rows' gradients; the other rows' stay."""
    hidden, head, t, w = loss_inputs(14, n, 500, 64, FP, ignored=0.0)
    clean = run_loss(hidden, head, t, w)
    bad = w.clone()
    bad[3], bad[9] = float("inf"), float("nan")
    dh = run_loss(hidden, head, t, bad)[2]
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[3] = rest[9] = False
    assert not torch.isfinite(dh[~rest]).any()
    # the largest finite weight, which P is divided by, is the same or leaves the same to 2 u a term
    assert torch.allclose(dh[rest], clean[2][rest], rtol=1e-5, atol=1e-9)
    only = torch.full_like(w, float("nan"))
    assert torch.isnan(run_loss(hidden, head, t, only)[2]).all()


@pytest.mark.parametrize("which", ["hidden", "head"])
def test_token_loss_one_gradient(which):
    from recurrent_memory_transformer_diag_b200 import token_loss_grad
    n, v, d = 200, 900, 128
    hidden, head, t, w = loss_inputs(6, n, v, d, BF)
    loss, lse, dh, dw = run_loss(hidden, head, t, w)
    if which == "hidden":
        x = torch.empty_like(hidden)
        token_loss_grad(hidden, head, t, lse, w, d_hidden=x)
        assert torch.equal(x, dh)
    else:
        x = torch.empty_like(head)
        token_loss_grad(hidden, head, t, lse, w, d_head=x)
        assert torch.equal(x, dw)


def test_token_loss_gradient_against_differences():
    """Central differences of the loss along a random direction.  The loss along a line
    is a sum of cumulant functions of a = max |u . w| at most: the third derivative is at
    most 2 a^3 a row, so the difference is within e^2 / 3 a^3 sum g, plus the losses' own
    error over e."""
    from recurrent_memory_transformer_diag_b200 import token_loss
    n, v, d = 50, 700, 64
    hidden, head, t, w = loss_inputs(8, n, v, d, FP)
    loss, lse, dh, dw = run_loss(hidden, head, t, w)
    g = gen(77)
    ok = (t >= 0).double()

    def total(h, hd):
        l, s = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        token_loss(h, hd, t, l, s)
        return float((l.double() * w.double() * ok).sum())

    e = 2.0 ** -6
    u = randn(g, n, d)
    a = float((u.double() @ head.double().t()).abs().max())
    noise = 64 * U * 20 * float((w.double() * ok).sum()) / e
    slope = (total(hidden + e * u, head) - total(hidden - e * u, head)) / (2 * e)
    assert abs(slope - float((dh.double() * u.double()).sum())) <= e * e / 3 * a ** 3 * float((w * ok).sum()) + noise
    u = randn(g, v, d) / math.sqrt(d)
    a = float((hidden.double() @ u.double().t()).abs().max())
    slope = (total(hidden, head + e * u) - total(hidden, head - e * u)) / (2 * e)
    assert abs(slope - float((dw.double() * u.double()).sum())) <= e * e / 3 * a ** 3 * float((w * ok).sum()) + noise


# ------------------------------------------------------------------ streams, graphs, together
def test_operators_on_another_stream_and_captured():
    """The whole chain on a side stream, then captured into a graph and replayed on
    other inputs: the same bits as calls one by one."""
    from recurrent_memory_transformer_diag_b200 import (embed, embed_grad, rms_norm, rms_norm_grad, token_loss,
                                                        token_loss_grad)
    n, v, d = 2500, 700, 128
    g = gen(12)
    s = {"table": randn(g, v, d).to(BF), "gain": (1 + 0.1 * randn(g, d)).to(BF),
         "ids": torch.randint(-1, v, (n,), generator=g, device="cuda"),
         "t": torch.randint(-1, v, (n,), generator=g, device="cuda"), "w": torch.full((n,), 1.0 / n, device="cuda")}

    def chain(stream=None):
        x, y = torch.empty(n, d, dtype=BF, device="cuda"), torch.empty(n, d, dtype=BF, device="cuda")
        r, loss, lse = (torch.empty(n, device="cuda") for _ in range(3))
        dy, dx, dt, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(s["table"]), torch.empty_like(s["gain"])
        embed(s["ids"], s["table"], x, scale=3.0, stream=stream)
        rms_norm(x, s["gain"], y, r, stream=stream)
        token_loss(y, s["table"], s["t"], loss, lse, stream=stream)
        token_loss_grad(y, s["table"], s["t"], lse, s["w"], dy, dt, stream=stream)
        rms_norm_grad(x, s["gain"], r, dy, dx, dg, stream=stream)
        embed_grad(s["ids"], dx, dt, scale=3.0, accumulate=True, stream=stream)
        return loss, lse, dx, dg, dt

    def same(a, b):
        torch.cuda.synchronize()
        return all(torch.equal(x, y) for x, y in zip(a, b))

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(side)
    assert same(got, want)
    got = chain(side.cuda_stream)      # a raw handle
    assert same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    other = randn(g, v, d).to(BF)
    s["table"].copy_(other)
    s["ids"].copy_(torch.randint(-1, v, (n,), generator=g, device="cuda"))
    want = chain()
    graph.replay()
    assert same(held, want)
    graph.replay()
    assert same(held, want)


def test_two_graphs_with_their_own_workspaces_replayed_side_by_side():
    from recurrent_memory_transformer_diag_b200 import token_loss, token_loss_grad
    n, v, d = 300, 2000, 64
    cases, graphs, outs, want = [], [], [], []
    for k in range(2):
        hidden, head, t, w = loss_inputs(20 + k, n, v, d, BF)
        cases.append((hidden, head, t, w))
        want.append(run_loss(hidden, head, t, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for hidden, head, t, w in cases:
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dh, dw = torch.empty_like(hidden), torch.empty_like(head)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            token_loss(hidden, head, t, loss, lse)
            token_loss_grad(hidden, head, t, lse, w, dh, dw)
        graphs.append(graph)
        outs.append((loss, lse, dh, dw))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_of_several_threads():
    """Calls of other sizes from other host threads, each on its own stream."""
    import threading
    cases = [loss_inputs(50 + k, n, v, d, dt) for k, (n, v, d, dt) in enumerate(
        [(3, 900, 2048, FP), (9, 700, 64, FP), (300, 1000, 128, BF), (40, 3000, 256, BF)])]
    want = [run_loss(*c) for c in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(c, expect):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = run_loss(*c)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, expect)):
                    wrong.append(c[0].shape)
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_offsets_past_32_bits():
    """Tables, hidden states and gradients of more than 2^31 elements."""
    from recurrent_memory_transformer_diag_b200 import embed, embed_grad, rms_norm, token_loss, token_loss_grad
    v, d = 300000, 8192
    g = gen(60)
    table = torch.zeros(v, d, dtype=BF, device="cuda")
    ids = torch.tensor([v - 1, 3, v - 2, 262144, 262145, -1, v], device="cuda")
    ok = ids[:5]
    table[ok] = randn(g, 5, d).to(BF)
    out = torch.empty(7, d, dtype=BF, device="cuda")
    embed(ids, table, out)
    assert torch.equal(out[:5], table[ok]) and (out[5:] == 0).all()
    n = 200                                       # sorted ids, and a table zeroed past 2^31 elements
    many = torch.cat([ok, torch.full((n - 5,), v - 1, device="cuda")])
    d_out = torch.ones(n, d, dtype=BF, device="cuda")
    grad = torch.full((v, d), 7.0, dtype=BF, device="cuda")
    embed_grad(many, d_out, grad)
    assert (grad[v - 1] == 196).all() and (grad[ok[1:]] == 1).all()
    grad[ok] = 0
    assert not grad.any()
    # a head of that size: the zero rows' logits are 0
    hidden = (randn(g, 70, d) / 32).to(BF)
    for rows in (3, 70):
        t = ok[torch.arange(rows, device="cuda") % 5].clone()
        h = hidden[:rows].contiguous()
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        token_loss(h, table, t, loss, lse)
        L = h.double() @ table[ok].double().t()
        want = torch.log(torch.exp(L).sum(1) + (v - 5))
        A = (h.double().abs() @ table[ok].double().abs().t()).max(1).values
        check(lse, want, logit_error(A, d, 1) + 1e-6 * want)
        w = torch.ones(rows, device="cuda")
        dh = torch.empty_like(h)
        grad.fill_(3.0)
        token_loss_grad(h, table, t, lse, w, dh, grad)
        P = torch.exp(L - want[:, None])
        P[torch.arange(rows, device="cuda"), torch.arange(rows, device="cuda") % 5] -= 1
        dw = P.t() @ h.double()
        mag = P.abs().t() @ h.double().abs()
        check(grad[ok], dw, mag * (half(BF) + 1e-4) + dw.abs() * half(BF))
        p0 = torch.exp(-want)[:, None] * h.double()   # any row of zeros
        for row in (0, 150000, 262143, 262146, v - 3):
            check(grad[row], p0.sum(0), p0.abs().sum(0) * (half(BF) + 1e-3) + p0.sum(0).abs() * half(BF))
        check(dh, P @ table[ok].double(), P.abs() @ table[ok].double().abs() * (half(BF) + 1e-4) + 1e-2 * half(BF)
              + (P @ table[ok].double()).abs() * half(BF))
    del grad
    y = torch.empty_like(table)
    gain = torch.ones(d, dtype=BF, device="cuda")
    rms_norm(table, gain, y, None, 1e-6)
    x = table[ok].double()
    want = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()
    check(y[ok], want, want.abs() * (half(BF) + 1e-5))


def test_given_workspace_and_status():
    from recurrent_memory_transformer_diag_b200 import token_loss, workspace_bytes, workspace_status
    n, v, d = 100, 500, 64
    hidden, head, t, w = loss_inputs(30, n, v, d, BF)
    size = workspace_bytes("token_loss", BF, n, d, v)
    ws = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    token_loss(hidden, head, t, loss, lse, workspace=ws[:size])
    workspace_status(ws)
    assert (ws[size:] == 255).all()      # nothing behind the size asked for
    assert torch.equal(loss, run_loss(hidden, head, t, w)[0])


@pytest.mark.parametrize("name", ["tiny", "small"])
def test_score_runs_ids_to_losses(name):
    """Armt.score: the losses of its embedding, forward, norm and loss, against the
    64-bit result from the forward's own hidden states; and streamed in two calls."""
    from recurrent_memory_transformer_diag_b200 import Armt, ArmtError, CONFIGS, make_weights
    cfg = CONFIGS[name]
    dt = BF if cfg.dtype == "bf16" else FP
    S, T, d, v = 4, cfg.seg_len, cfg.d_model, 515
    g = gen(40)
    table = randn(g, v, d).to(dt)
    head = (randn(g, v, d) / math.sqrt(d)).to(dt)
    gain = (1 + 0.1 * randn(g, d)).to(dt)
    ids = torch.randint(0, v, (S * T,), generator=g, device="cuda")
    targets = torch.cat([ids[1:], ids.new_full((1,), -1)])
    state = lambda: (torch.zeros(cfg.n_layers, d, cfg.phi_dim, device="cuda"),  # noqa: E731
                     torch.zeros(cfg.n_layers, cfg.phi_dim, device="cuda"))
    with Armt(cfg, max_segments=S) as m:
        m.load_weights(make_weights(cfg))
        A, z = state()
        loss = torch.empty(S * T, device="cuda")
        m.score(ids, targets, S, T, table, head, gain, loss, A, z)
        m.device_status()
        hidden = torch.empty(S * T, d, dtype=dt, device="cuda")
        A2, z2 = state()
        m.forward(table[ids].contiguous(), S, T, hidden, A2, z2)
        assert torch.equal(A, A2) and torch.equal(z, z2)
        H = hidden.double()
        y = (H / (H.square().mean(1, keepdim=True) + cfg.rms_eps).sqrt() * gain.double()).to(dt)
        _, rl, rloss, Amax, _ = loss_reference(y, head, targets, 1.0)
        # the norm's own rounding may fall the other way: one step of the type in some elements
        check(loss, rloss, Amax * (4 * half(dt) + 128 * U) + 1e-4 * U, "score")
        # two calls of two segments, the state carried
        A3, z3 = state()
        parts = []
        for k in range(2):
            p = torch.empty(2 * T, device="cuda")
            sl = slice(k * 2 * T, (k + 1) * 2 * T)
            m.score(ids[sl], targets[sl], 2, T, table, head, gain, p, A3, z3, carry_state=True)
            parts.append(p)
        torch.cuda.synchronize()
        assert torch.equal(torch.cat(parts), loss)
        # a wrong tensor is refused before the state changes
        good = {"ids": ids, "targets": targets, "table": table, "head": head, "gain": gain, "loss": loss}
        for name, bad in (("ids", ids[1:]), ("targets", targets.float()), ("table", table[:, :8].contiguous()),
                          ("head", head.to(FP if dt == BF else BF)), ("gain", gain[1:]), ("loss", loss[1:]),
                          ("loss", A3.view(-1)[:S * T])):
            q = {**good, name: bad}
            before = A3.clone(), z3.clone()
            with pytest.raises(ArmtError):
                m.score(q["ids"], q["targets"], S, T, q["table"], q["head"], q["gain"], q["loss"], A3, z3)
            torch.cuda.synchronize()
            assert torch.equal(A3, before[0]) and torch.equal(z3, before[1])


@pytest.mark.parametrize("rows", [4, 40, 200])
def test_bounded_waits_of_the_loss(rows):
    """Copies that never come: the waits run out after about a second, the status and a
    NaN loss say so, and the next call (in this process, on this device) is right."""
    import time
    from recurrent_memory_transformer_diag_b200.armt import STATUS, lib
    t0 = time.time()
    status = lib().armt_test_loss_wait(rows, torch.cuda.current_stream().cuda_stream)
    assert STATUS[status] == "ARMT_ERR_DEVICE_TIMEOUT" and time.time() - t0 < 20
    hidden, head, t, w = loss_inputs(rows, rows, 700, 128, BF)
    check_loss(hidden, head, t, w, 1.0, run_loss(hidden, head, t, w))


# ------------------------------------------------------------------ refusals
def _refusals():
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    n, v, d = 6, 20, 64
    base = {"x": z(n, d), "y": z(n, d), "dy": z(n, d), "dx": z(n, d), "w": z(v, d), "dw": z(v, d), "gain": z(d),
            "dg": z(d), "f": z(n, dt=FP), "f2": z(n, dt=FP), "f3": z(n, dt=FP),
            "i": torch.zeros(n, dtype=torch.int64, device="cuda")}
    calls = {
        "embed": lambda o, b: o.embed(b["i"], b["w"], b["y"]),
        "embed_grad": lambda o, b: o.embed_grad(b["i"], b["dy"], b["dw"]),
        "rms_norm": lambda o, b: o.rms_norm(b["x"], b["gain"], b["y"], b["f"]),
        "rms_norm_grad": lambda o, b: o.rms_norm_grad(b["x"], b["gain"], b["f"], b["dy"], b["dx"], b["dg"]),
        "token_loss": lambda o, b: o.token_loss(b["x"], b["w"], b["i"], b["f"], b["f2"]),
        "token_loss_grad": lambda o, b: o.token_loss_grad(b["x"], b["w"], b["i"], b["f"], b["f2"], b["dx"], b["dw"]),
    }
    shift = lambda *s: torch.zeros(math.prod(s) + 1, dtype=BF, device="cuda")[1:].view(*s)  # noqa: E731
    return base, calls, [
        ("embed", "w", z(v, d, dt=torch.float16)), ("embed", "w", z(v, d).t()), ("embed", "w", shift(v, d)),
        ("embed", "i", z(n)), ("embed", "i", z(2 * n).long()[::2]), ("embed", "y", z(n, d, dt=FP)),
        ("embed", "y", z(n + 1, d)), ("embed", "y", base["w"][:n]), ("embed", "w", z(v, 60)), ("embed", "y", z(n, d).cpu()),
        ("embed_grad", "dw", z(v, d + 8)), ("embed_grad", "dw", z(v * d)), ("embed_grad", "i", z(n + 1).long()),
        ("embed_grad", "dy", z(n, 2 * d)[:, :d]), ("embed_grad", "dw", base["dy"]), ("embed_grad", "dw", None),
        ("rms_norm", "gain", z(d, dt=FP)), ("rms_norm", "f", z(n)), ("rms_norm", "y", base["x"].view(-1)[d:].new_zeros(n, d + 8)),
        ("rms_norm", "x", z(n, d, 1)), ("rms_norm", "gain", z(d + 8)), ("rms_norm", "y", None),
        ("rms_norm_grad", "dx", base["gain"].expand(n, d)), ("rms_norm_grad", "dg", base["x"][0]),
        ("rms_norm_grad", "f", z(n + 1, dt=FP)), ("rms_norm_grad", "dy", z(n, d, dt=FP)),
        ("token_loss", "w", z(v, d, dt=FP)), ("token_loss", "i", z(n, 1).long()), ("token_loss", "f", z(n)),
        ("token_loss", "f2", base["f"]), ("token_loss", "x", shift(n, d)), ("token_loss", "w", z(v, d + 8)),
        ("token_loss_grad", "dx", base["x"]), ("token_loss_grad", "dw", base["w"]), ("token_loss_grad", "f2", z(n)),
        ("token_loss_grad", "dw", z(v, d, dt=FP)), ("token_loss_grad", "dx", z(n, d).t()),
        ("token_loss_grad", "i", z(n).to(torch.int16)),
    ]


@pytest.mark.parametrize("k", range(38))
def test_wrappers_refuse(k):
    """One wrong tensor at a time: an error, and nothing is written."""
    from recurrent_memory_transformer_diag_b200 import ArmtError, operators as ops
    base, calls, wrong = _refusals()
    assert len(wrong) == 38
    op, name, t = wrong[k]
    before = {q: u.clone() for q, u in base.items()}
    with pytest.raises(ArmtError) as e:
        calls[op](ops, {**base, name: t})
    assert e.value.status in (1, 7)
    torch.cuda.synchronize()
    assert all(torch.equal(before[q], base[q]) for q in base)


def test_wrappers_refuse_workspaces():
    from recurrent_memory_transformer_diag_b200 import ArmtError, embed_grad, token_loss, workspace_bytes
    n, v, d = 200, 300, 64
    hidden, head, t, w = loss_inputs(1, n, v, d, BF)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    size = workspace_bytes("token_loss", BF, n, d, v)
    for ws in (torch.empty(size - 1, dtype=torch.uint8, device="cuda"), torch.empty(size, dtype=torch.uint8),
               torch.empty(size // 4 + 1, device="cuda"), torch.empty(size + 8, dtype=torch.uint8, device="cuda")[8:],
               torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2], 5):
        with pytest.raises(ArmtError):
            token_loss(hidden, head, t, loss, lse, workspace=ws)
    out = torch.empty(v, d, dtype=BF, device="cuda")
    size = workspace_bytes("embed_grad", BF, n, d, v)
    assert size > 0
    with pytest.raises(ArmtError):
        embed_grad(t, hidden, out, workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ArmtError):   # results inside the workspace
        ws = torch.empty(size + v * d * 2, dtype=torch.uint8, device="cuda")
        embed_grad(t, hidden, ws[:v * d * 2].view(BF).view(v, d), workspace=ws)


# ------------------------------------------------------------------ logits far below zero
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("at", [-100.0, -200.0])
@pytest.mark.parametrize("n,v,d", [(40, 300, 64), (65, 300, 64), (65, 1025, 64), (300, 300, 136), (300, 1025, 64),
                                   (3000, 1000, 64)])
def test_token_loss_logits_far_below_zero(n, v, d, at, dtype):
    """Every logit near `at`, so that exp(0 - lse) is past fp32: columns behind a vocabulary that
    ends inside a tile, whose logits would be 0, count nowhere."""
    hidden, head, t, w = loss_inputs(n + v, n, v, d, dtype)
    head[:, 0], hidden[:, 0] = 4.0, at / 4
    got = run_loss(hidden, head, t, w)
    assert all(torch.isfinite(x).all() for x in got) and float(got[1].min()) < at + 40
    check_loss(hidden, head, t, w, 1.0, got)


@pytest.mark.parametrize("n,v,d,dtype", [(8192, 17000, 64, BF), (4100, 11003, 64, FP)])
def test_token_loss_logits_far_below_zero_in_pieces(n, v, d, dtype):
    """The same with the gradient in two pieces of the vocabulary, the second ragged."""
    hidden, head, t, w = loss_inputs(n + 1, n, v, d, dtype)
    head[:, 0], hidden[:, 0] = 4.0, -30.0
    got = run_loss(hidden, head, t, w)
    assert all(torch.isfinite(x).all() for x in got)
    check_loss(hidden, head, t, w, 1.0, got)


# ------------------------------------------------------------------ P and lse from the same logits
@pytest.mark.parametrize("n,v,d", [(1, 1000, 2048), (3, 1000, 8192), (40, 1000, 2048), (40, 1000, 8192), (200, 1000, 2048),
                                   (200, 1000, 8192), (2000, 1000, 4096)])
def test_token_loss_gradient_of_sure_rows(n, v, d):
    """Targets of probability near 1 (1 - p about 2e-4, logits of 16, many columns): p - 1 is a
    small difference.  Where P is made of the very logits that its lse is made of, their errors
    el (as in logit_error) only change 1 - p by its el-th part; what is left is the rounding of
    lse, of its sum and of the exponential."""
    g = gen(n + d)
    head = (randn(g, v, d) / math.sqrt(d)).to(BF)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    hidden = (randn(g, n, d) + 16 * head[t].float()).to(BF)
    w = torch.ones(n, device="cuda")
    loss, lse, dh, dw = run_loss(hidden, head, t, w)
    L, rl, _, A, _ = loss_reference(hidden, head, t, 1.0)
    el = logit_error(A, d, 1) + L.abs().max(1).values * U
    es = (16 + 64 + v / 256) * U + 4 * U * (rl.abs() + 1)      # as in check_loss: sum and logarithm
    P = torch.exp(L - rl[:, None])
    at = t[:, None]
    Q = P.scatter_add(1, at, torch.full_like(P[:, :1], -1.0))
    gap = (L - rl[:, None]).abs()
    rest = -Q.gather(1, at)[:, 0]
    assert float(rest.median()) < 1e-3
    # the others: exp(l - lse) relative; the target: its complement
    ep = P * (2 * el + es + 8 * U)[:, None] + P * gap * 3 * U
    ep.scatter_(1, at, (rest * 2 * el + es + 8 * U)[:, None])
    ep = ep + Q.abs() * (2.0 ** -16 if n <= 64 else half(BF))   # two terms of P, or one
    W = head.double()
    want = Q @ W
    check(dh, want, ep @ W.abs() + Q.abs() @ W.abs() * ((v / 16 + 2) * 4 + 24) * U + want.abs() * half(BF) + 1e-38, "d_hidden")


def test_token_loss_head_gradient_of_many_rows():
    """Sums over 262144 rows of one sign: no bias of a long accumulator.  Logits of 0 and 512
    entries make P of every entry but the target exactly 2^-9, so that the only errors are those
    of the sum: an accumulator of K = 8192 at most (512 instructions, 2 u in the instruction and
    2 u in the accumulator), 32 of them added to nearest, the scale, and the last rounding (half
    of the step where the result lies)."""
    from recurrent_memory_transformer_diag_b200 import token_loss, token_loss_grad
    n, v, d = 262144, 512, 8192
    g = gen(71)
    hidden = (1 + torch.rand(n, d, generator=g, device="cuda", dtype=BF)).mul_(
        torch.linspace(1, 2, d, device="cuda").to(BF))
    head = torch.zeros(v, d, dtype=BF, device="cuda")
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    token_loss(hidden, head, t, loss, lse)
    dw = torch.empty_like(head)
    token_loss_grad(hidden, head, t, lse, torch.ones(n, device="cuda"), d_head=dw)
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for part in hidden.split(8192):
        want += part.double().sum(0)
    want *= 2.0 ** -9
    step = torch.exp2(torch.floor(torch.log2(want))) * 2.0 ** -7
    check(dw[1:], want.expand(v - 1, d), (step / 2 + want * (512 * 4 + 32 + 2) * U).expand(v - 1, d))


# ------------------------------------------------------------------ Armt.score refuses before it changes the state
def score_inputs(name="small", v=515):
    from recurrent_memory_transformer_diag_b200 import CONFIGS
    cfg = CONFIGS[name]
    dt, n, d = BF if cfg.dtype == "bf16" else FP, 2 * cfg.seg_len, cfg.d_model
    g = gen(41)
    table, head = randn(g, v, d).to(dt), (randn(g, v, d) / math.sqrt(d)).to(dt)
    ids = torch.randint(0, v, (n,), generator=g, device="cuda")
    state = randn(g, cfg.n_layers, d, cfg.phi_dim) * 1e-2, torch.rand(cfg.n_layers, cfg.phi_dim, generator=g, device="cuda")
    return cfg, dict(ids=ids, targets=ids.roll(-1), n_segments=2, seg_len=cfg.seg_len, table=table, head=head,
                     gain=torch.ones(d, dtype=dt, device="cuda"), loss=torch.zeros(n, device="cuda"), A=state[0],
                     z=state[1], carry_state=True)


def off_by_one(x):
    """The same numbers, dense, two or four bytes off a 16-byte boundary."""
    y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
    return y.copy_(x)


@pytest.mark.parametrize("name", ["tiny", "small"])
def test_score_refuses_before_the_state_changes(name, monkeypatch):
    """What the norm and the loss would refuse after the forward, or could not allocate:
    the streamed state and the losses stay, so that the segment can be scored again."""
    from recurrent_memory_transformer_diag_b200 import Armt, ArmtError, make_weights, workspace_bytes, workspace_status
    cfg, call = score_inputs(name)
    n, d, v = len(call["ids"]), cfg.d_model, len(call["head"])
    size = workspace_bytes("token_loss", call["head"].dtype, n, d, v)
    space = torch.empty(size, dtype=torch.uint8, device="cuda")
    head_size = call["head"].element_size()
    shared = torch.zeros(size + v * d * head_size, dtype=torch.uint8, device="cuda")
    with Armt(cfg, max_segments=2) as m:
        m.load_weights(make_weights(cfg))
        kept = [(k, call[k], call[k].clone()) for k in ("A", "z", "loss", "head", "table")]

        def untouched():
            torch.cuda.synchronize()
            return all(torch.equal(a, b) for _, a, b in kept)
        for wrong in (dict(head=off_by_one(call["head"])), dict(gain=off_by_one(call["gain"])),
                      dict(table=off_by_one(call["table"])), dict(logit_scale=float("inf")),
                      dict(logit_scale=float("nan")), dict(logit_scale=1e300), dict(embed_scale=float("nan")),
                      dict(n_segments=3), dict(workspace=space[:-1]), dict(workspace=space.cpu()), dict(workspace=7),
                      dict(workspace=shared, head=shared[:v * d * head_size].view(call["head"].dtype).view(v, d))):
            with pytest.raises(ArmtError):
                m.score(**{**call, **wrong})
            assert untouched(), wrong.keys()
        # no memory left for the loss
        import recurrent_memory_transformer_diag_b200.operators as ops
        real = torch.empty

        def empty(*a, **k):
            if k.get("dtype") is torch.uint8:
                raise torch.cuda.OutOfMemoryError("no workspace")
            return real(*a, **k)
        monkeypatch.setattr(ops.torch, "empty", empty)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            m.score(**call)
        assert untouched()
        monkeypatch.undo()
        # the caller's own workspace: the same losses, and its status can be read
        A, z = call["A"].clone(), call["z"].clone()
        m.score(**call, workspace=space)
        workspace_status(space)
        want = call["loss"].clone()
        assert float(want.min()) > 0 and not torch.equal(A, call["A"])
        m.score(**{**call, "A": A, "z": z})
        torch.cuda.synchronize()
        assert torch.equal(call["loss"], want) and torch.equal(A, call["A"]) and torch.equal(z, call["z"])


def test_score_refuses_another_device_than_the_context_s(monkeypatch):
    """A context's weights and workspaces are on one device; tensors of another are refused
    (here by a context that takes itself for one of the next device)."""
    from recurrent_memory_transformer_diag_b200 import Armt, ArmtError, make_weights
    cfg, call = score_inputs("tiny")
    with Armt(cfg, max_segments=2) as m:
        m.load_weights(make_weights(cfg))
        assert m.device_index == torch.cuda.current_device()
        before = call["A"].clone()
        monkeypatch.setattr(m, "device_index", m.device_index + 1)
        with pytest.raises(ArmtError, match="device"):
            m.score(**call)
        torch.cuda.synchronize()
        assert torch.equal(call["A"], before)


@pytest.mark.parametrize("op,name", [("embed_grad", "d_out"), ("embed_grad", "ids"), ("rms_norm_grad", "x"),
                                     ("rms_norm_grad", "gain"), ("rms_norm_grad", "rstd"), ("rms_norm_grad", "dy"),
                                     ("token_loss", "hidden"), ("token_loss", "head"), ("token_loss", "targets"),
                                     ("token_loss_grad", "hidden"), ("token_loss_grad", "head"),
                                     ("token_loss_grad", "targets"), ("token_loss_grad", "lse"),
                                     ("token_loss_grad", "d_loss")])
def test_wrappers_refuse_inputs_inside_the_workspace(op, name):
    """A workspace is written while the inputs are read: one input in it is refused, nothing is written."""
    import recurrent_memory_transformer_diag_b200 as armt
    n, v, d = 200, 300, 64
    hidden, head, t, w = loss_inputs(1, n, v, d, BF)
    t.clamp_(min=0)
    new = lambda x: torch.zeros_like(x)  # noqa: E731
    ins, outs = {
        "embed_grad": (dict(ids=t, d_out=hidden), dict(d_table=new(head))),
        "rms_norm_grad": (dict(x=hidden, gain=head[0].clone(), rstd=w, dy=hidden.clone()),
                          dict(dx=new(hidden), d_gain=new(head[0]))),
        "token_loss": (dict(hidden=hidden, head=head, targets=t), dict(loss=new(w), lse=new(w))),
        "token_loss_grad": (dict(hidden=hidden, head=head, targets=t, lse=w, d_loss=w.clone()),
                            dict(d_hidden=new(hidden), d_head=new(head))),
    }[op]
    size = armt.workspace_bytes(op, BF, n, d, v)
    space = torch.zeros(size + ins[name].nbytes, dtype=torch.uint8, device="cuda")
    at = (size // 2 + 255) // 256 * 256      # the input in the middle of what the operator would write
    part = space[at:at + ins[name].nbytes].view(ins[name].dtype).view(ins[name].shape).copy_(ins[name])
    before = space.clone()
    with pytest.raises(armt.ArmtError, match="workspace overlaps"):
        getattr(armt, op)(**{**ins, name: part}, **outs, workspace=space)
    torch.cuda.synchronize()
    assert torch.equal(space, before) and all((x == 0).all() for x in outs.values())
    getattr(armt, op)(**ins, **outs, workspace=space)     # apart: fine
    torch.cuda.synchronize()


def test_results_count_as_written_in_place():
    """Autograd notices that a tensor it has kept was overwritten by an operator (as by any
    in-place operation), and inputs do not count as written."""
    from recurrent_memory_transformer_diag_b200 import (embed, embed_grad, rms_norm, rms_norm_grad, token_loss,
                                                        token_loss_grad)
    n, v, d = 12, 40, 64
    hidden, head, t, w = loss_inputs(70, n, v, d, FP)
    gain, f = torch.ones(d, device="cuda"), lambda: torch.empty(n, device="cuda")
    out = lambda x: torch.empty_like(x)  # noqa: E731
    calls = [(embed, (t, head), (out(hidden),)), (embed_grad, (t, hidden), (out(head),)),
             (rms_norm, (hidden, gain), (out(hidden), f())),
             (rms_norm_grad, (hidden, gain, w, hidden), (out(hidden), out(gain))),
             (token_loss, (hidden, head, t), (f(), f())),
             (token_loss_grad, (hidden, head, t, w, w), (out(hidden), out(head)))]
    for fn, ins, outs in calls:
        before = [x._version for x in ins + outs]
        fn(*ins, *outs)
        after = [x._version for x in ins + outs]
        k = len(ins)
        assert after[:k] == before[:k] and all(a > b for a, b in zip(after[k:], before[k:])), fn.__name__
    x = torch.ones(n, d, device="cuda")
    p = torch.ones(n, d, device="cuda", requires_grad=True)
    y = (p * x).sum()          # keeps x
    rms_norm(x, gain, x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_raw_handle_of_the_default_stream():
    """Handle 0 is the default stream (what current_stream().cuda_stream gives there): a call on it
    comes after what is queued there and before what follows."""
    from recurrent_memory_transformer_diag_b200 import rms_norm
    assert torch.cuda.current_stream().cuda_stream == 0
    x = torch.zeros(256, 64, device="cuda")
    gain, y, z = torch.ones(64, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    rms_norm(x, gain, y)
    torch.cuda.synchronize()
    for _ in range(4):
        x.zero_()
        torch.cuda._sleep(20_000_000)      # some 10 ms
        x.fill_(2.0)
        rms_norm(x, gain, y, None, 0.0, stream=torch.cuda.current_stream().cuda_stream)
        z.copy_(y)
        y.zero_()
        torch.cuda.synchronize()
        assert (z == 1).all() and (y == 0).all()


@pytest.mark.parametrize("n", [40, 300, 3000])
def test_loss_on_the_default_stream_s_handle(n):
    hidden, head, t, w = loss_inputs(80, n, 3000, 64, BF)
    want = run_loss(hidden, head, t, w)
    from recurrent_memory_transformer_diag_b200 import token_loss, token_loss_grad
    for _ in range(10):
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dh, dw = torch.empty_like(hidden), torch.empty_like(head)
        token_loss(hidden, head, t, loss, lse, stream=0)
        token_loss_grad(hidden, head, t, lse, w, dh, dw, stream=0)
        got = loss.clone(), lse.clone(), dh.clone(), dw.clone()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_inputs_behind_what_is_used_of_a_workspace():
    """One arena for all: inputs behind the bytes that the operator asks for are no overlap."""
    from recurrent_memory_transformer_diag_b200 import token_loss, workspace_bytes
    n, v, d = 100, 300, 64
    hidden, head, t, w = loss_inputs(90, n, v, d, BF)
    size = (workspace_bytes("token_loss", BF, n, d, v) + 255) // 256 * 256
    arena = torch.zeros(size + hidden.nbytes, dtype=torch.uint8, device="cuda")
    inside = arena[size:].view(BF).view(n, d).copy_(hidden)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    token_loss(inside, head, t, loss, lse, workspace=arena)
    assert torch.equal(inside, hidden) and torch.equal(loss, run_loss(hidden, head, t, w)[0])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [3, 40, 200])
def test_token_loss_entries_masked_by_the_lowest_value(n, dtype):
    """Vocabulary entries whose logit is the type's lowest number (whole tiles among them) have no
    part in the loss and no gradient: the same as without them, to the order of the sums."""
    v, d = 900, 64
    hidden, head, t, w = loss_inputs(95, n, v, d, dtype, ignored=0.0)
    masked = torch.rand(v, generator=gen(96), device="cuda") < 0.5
    masked[256:640] = True
    masked[t] = False
    hidden[:, 0], head[:, 0] = 1.0, 0.0
    head[masked, 0] = torch.finfo(dtype).min
    got = run_loss(hidden, head, t, w)
    keep = (~masked).nonzero()[:, 0]
    place = torch.zeros(v, dtype=torch.int64, device="cuda")
    place[keep] = torch.arange(len(keep), device="cuda")
    few = head[keep].contiguous()
    want = run_loss(hidden, few, place[t], w)
    check_loss(hidden, few, place[t], w, 1.0, (*got[:3], got[3][keep].contiguous()))
    assert (got[3][masked] == 0).all() and float((got[0] - want[0]).abs().max()) < 64 * U * float(want[1].abs().max() + 1)
