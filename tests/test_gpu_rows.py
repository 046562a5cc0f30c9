"""The feature-row operators on the GPU against plain 64-bit implementations.

Tolerances count roundings (u: half a step of the output type, 2^-24, 2^-11, 2^-8).  A sum of m
terms in fp32, in any order, is off by at most (m - 1) 2^-24 times the sum of their magnitudes.
8-bit rows: q8_pack is compared bit for bit; where the rows were computed first, a value is off by
its own error plus e4m3's half step, 2^-4 of the value, or 2^-10 of the scale, which is below
2 amax / 448 (and at least 2^-126).
"""
import threading

import numpy as np
import pytest
import torch

import oracle
from tests.util import rand_coords

pytestmark = pytest.mark.gpu

scv = pytest.importorskip("sparse_convolution_voxel_b200")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def _rand(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def _within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape and bool((err <= bound).all()), \
        f"{what}: worst {float((err / bound.clamp(min=1e-300)).max()):.3g} times the bound"


# --------------------------------------------------------------------------- 8-bit rows
def plain_q8(x):
    """(e4m3 bytes, scale bytes) of x by the format's arithmetic, in 64 bits on the host."""
    v = x.double().cpu().numpy()
    n, c = v.shape
    g = -(-c // 32)
    fine = np.isfinite(v)
    w = np.zeros((n, g * 32))
    w[:, :c] = np.where(fine, v, 0.0)
    amax = np.abs(w).reshape(n, g, 32).max(2)
    e = np.full((n, g), 1, np.int64)
    pos = amax > 0
    m, k = np.frexp(amax[pos] / 448.0)          # (1/2, 1] 2^k once powers of two are moved down
    e[pos] = np.maximum(1, np.where(m == 0.5, k - 1, k) + 127)
    u = w / np.ldexp(1.0, np.repeat(e, 32, 1) - 127)
    _, f = np.frexp(np.abs(u))
    step = np.maximum(f - 1, -6) - 3
    u = np.ldexp(np.rint(np.ldexp(u, -step)), step)[:, :c]
    q = torch.from_numpy(np.where(fine, u, np.nan)).float().to(torch.float8_e4m3fn)
    return q, torch.from_numpy(e).to(torch.uint8)


def values_q8(r):
    """The values of 8-bit rows in 64 bits, on their device."""
    s = torch.ldexp(torch.ones(r.scale.shape, dtype=torch.float64, device=r.scale.device), r.scale.int() - 127)
    return r.q.double() * s.repeat_interleave(32, 1)[:, :r.q.shape[1]]


def _check_q8(r, y, own, what):
    """8-bit rows r of values y (64 bits) that were computed with relative error `own` before."""
    n, c = y.shape
    pad = torch.nn.functional.pad(y.abs(), (0, -c % 32)).view(n, -1, 32).amax(2)
    scale = (2 * (1 + own) * pad / 448.0).clamp(min=2.0 ** -126).repeat_interleave(32, 1)[:, :c]
    _within(values_q8(r), y, (2.0 ** -4 * (1 + own) + own) * y.abs() + 2.0 ** -10 * scale, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", [(1, 8), (3, 16), (130, 32), (257, 40), (33, 72), (1000, 128), (5, 1000), (2, 16384),
                                 (61, 256), (64, 264)])
def test_pack_is_the_format_bit_for_bit(dtype, n, c):
    x = _rand(n + c, n, c) * torch.exp(2 * _rand(c, c))
    x = x.to(dtype)
    r = scv.q8_pack(x)
    q, s = plain_q8(x)
    assert torch.equal(r.scale.cpu(), s)
    assert torch.equal(r.q.view(torch.uint8).cpu(), q.view(torch.uint8))
    for to in DTYPES:
        v = scv.q8_unpack(r, to)
        want = values_q8(r)
        if to == torch.float16:
            want = want.clamp(-65504.0, 65504.0)
        assert torch.equal(v, want.to(to)), to


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_at_the_edges(dtype):
    """Groups of zeros, of the smallest and the largest values, at the powers of two and at 448 times one, at ties,
    with infinities and NaN among finite values, and with nothing finite."""
    fi = torch.finfo(dtype)
    x = torch.zeros(12, 72, dtype=torch.float64)
    x[1] = fi.max
    x[2] = -fi.max
    x[3] = fi.smallest_normal
    x[4, ::3] = float(torch.tensor(fi.smallest_normal).to(dtype)) * fi.eps      # the smallest subnormal
    x[5] = torch.linspace(-448, 448, 72)
    x[6] = 448.0
    x[7] = 448.0 + 448.0 * 2 * fi.eps                                           # the next value: the next scale
    x[8] = 1.0 + torch.arange(72) / 16.0                                        # ties between e4m3 values
    x[9] = 3.0
    x[9, 5], x[9, 40], x[9, 70] = float("inf"), float("-inf"), float("nan")
    x[10] = float("nan")
    x[11] = float("inf")
    x = x.to(dtype)
    r = scv.q8_pack(x.cuda())
    q, s = plain_q8(x)
    assert torch.equal(r.scale.cpu(), s)
    nan = ~torch.isfinite(x)
    got = r.q.cpu()
    assert bool(torch.isnan(got.float())[nan].all()) and bool(torch.isfinite(got.float())[~nan].all())
    assert torch.equal(got.view(torch.uint8)[~nan], q.view(torch.uint8)[~nan])
    half = scv.q8_unpack(r, torch.float16).cpu()
    assert bool(torch.isfinite(half)[~nan].all()), "fp16 is held at its largest value"
    assert torch.equal(torch.isnan(half), nan)


# --------------------------------------------------------------------------- embedding
def _ids(seed, n, vocab, dtype, pad=-1, share=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = (vocab * torch.rand(n, generator=g) ** 3).long().clamp(max=vocab - 1)
    ids[torch.rand(n, generator=g) < share] = pad
    return ids.to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,vocab,c", [(1, 1, 8), (7, 50, 16), (300, 1000, 64), (65, 9, 136), (1000, 5000, 256),
                                       (33, 77, 1032), (5, 3, 16384)])
def test_lookup(dtype, idt, n, vocab, c):
    ids, table = _ids(n, n, vocab, idt), _rand(c, vocab, c, dtype=dtype)
    scale = c ** 0.5
    st = scv.new_status()
    y = scv.embed_fwd(ids, table, scale, d_status=st)
    scv.check_status(st)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    ref = torch.where((ids >= 0)[:, None], table[ids.long().clamp(min=0)].double() * s32, 0.0)
    _within(y, ref, (UNIT[dtype] + 2.0 ** -24) * ref.abs() + TINY[dtype], "lookup")


@pytest.mark.parametrize("n,vocab,c", [
    (0, 5, 16), (1, 1, 8), (1, 300, 64), (37, 1, 128), (2000, 1, 64), (513, 40, 24), (2049, 2, 256),
    (5000, 700, 128), (5000, 100000, 8), (20000, 1 << 10, 64), (20000, 3000000, 8), (4096, 64, 512),
    (3000, 17, 1032), (70000, 300, 32), (150000, 5, 128), (4096, 255, 8), (4097, 256, 8), (8191, 70000, 16),
    (65536, 300, 8), (65537, 40000, 8), (33000, 1, 16), (5000, 1100000, 8), (4100, 262144, 8), (4100, 262145, 8),
    (0, 40000, 128), (0, 1100000, 8), (100, 700, 8192), (5000, 700, 8192), (4097, 260, 16384), (300000, 50000, 64),
])
@pytest.mark.parametrize("dtype,idt", [(torch.float32, torch.int32), (torch.bfloat16, torch.int64)])
def test_lookup_gradient(n, vocab, c, dtype, idt):
    """Few and many tokens, tokens with most of the rows and with none, one to three digits of the sort."""
    ids, dy = _ids(n + vocab, n, vocab, idt), _rand(n + c, n, c, dtype=dtype)
    scale, st = 3.0, scv.new_status()
    out = torch.full((vocab, c), float("nan"), device="cuda")
    dt = scv.embed_wgrad(ids, dy, vocab, scale, d_status=st, out=out)
    scv.check_status(st)
    have = ids >= 0
    at = ids[have].long()
    ref = torch.zeros(vocab, c, dtype=torch.float64, device="cuda").index_add_(0, at, dy[have].double())
    mag = torch.zeros(vocab, c, dtype=torch.float64, device="cuda").index_add_(0, at, dy[have].double().abs())
    count = torch.bincount(at, minlength=vocab).double()[:, None]
    _within(dt, ref * scale, (count + 2) * 2.0 ** -24 * mag * scale, "gradient")
    again = scv.embed_wgrad(ids, dy, vocab, scale)
    assert torch.equal(dt, again), "the bits depend on timing"


def test_lookup_padding_and_bad_ids():
    """A padding id in the middle of the vocabulary has no row; ids outside it are flagged and have none either."""
    table, dy = _rand(1, 20, 64), _rand(2, 10, 64)
    ids = torch.tensor([3, 7, 7, 0, 19, 3, 7, 5, 5, 1], dtype=torch.int64).cuda()
    st = scv.new_status()
    y, dt = scv.embed_fwd(ids, table, pad_id=7, d_status=st), scv.embed_wgrad(ids, dy, 20, pad_id=7, d_status=st)
    scv.check_status(st)
    assert not y[ids == 7].any() and not dt[7].any()
    assert torch.equal(y[ids != 7], table[ids[ids != 7]])
    assert torch.equal(dt[5], dy[7] + dy[8])
    bad = ids.clone()
    bad[0], bad[1], bad[2] = 20, -1, 1 << 40
    for f in (lambda s: scv.embed_fwd(bad, table, pad_id=7, d_status=s),
              lambda s: scv.embed_wgrad(bad, dy, 20, pad_id=7, d_status=s)):
        st = scv.new_status()
        out = f(st)
        with pytest.raises(scv.LatticeError, match="LAT_ERR_BAD_ID"):
            scv.check_status(st)
        assert bool(torch.isfinite(out).all())
    good = torch.tensor([3, 4, 5, 7, 8, 9]).cuda()  # the rows with a token
    ref = torch.zeros_like(dt).index_add_(0, bad[good[good != 6]], dy[good[good != 6]])
    ref[7] = 0
    assert torch.allclose(out, ref, rtol=1e-6, atol=0)


def test_rows_without_a_token_are_not_read():
    """Padded rows come out as 0 whatever the scale is, and what their dy holds counts nowhere."""
    table, dy = _rand(1, 20, 64), _rand(2, 5000, 64)
    ids = _ids(3, 5000, 20, torch.int64)
    pad = torch.arange(5000, device="cuda") % 3 == 0
    ids[pad] = -1
    want = scv.embed_wgrad(ids, torch.where(pad[:, None], 0.0, dy), 20)
    dy[pad] = float("nan")
    assert torch.equal(scv.embed_wgrad(ids, dy, 20), want)
    for scale in (float("inf"), float("nan"), -1.0):
        assert not scv.embed_fwd(ids, table, scale)[pad].view(torch.int32).any()


def test_lookup_gradient_without_a_token():
    dy = _rand(4, 5000, 128)
    ids = torch.full((5000,), -1, dtype=torch.int32, device="cuda")
    assert not scv.embed_wgrad(ids, dy, 300).any()


# --------------------------------------------------------------------------- RMS norm
SHAPES = [(1, 8), (5, 16), (33, 40), (300, 64), (17, 72), (1000, 128), (129, 200), (70, 256), (31, 264), (9, 512),
          (40, 520), (3, 1024), (7, 2056), (4, 4096), (5, 5120), (3, 8192), (2, 16384)]
OWN = 2.0 ** -18  # of the forward pass before the rounding: 64 fp32 roundings


def plain_norm(x, res, w, eps):
    h = x.double() if res is None else x.double() + res.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    y = h * rstd[:, None]
    return h, rstd, y if w is None else y * w.double()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", SHAPES)
@pytest.mark.parametrize("with_res", [False, True])
def test_norm(dtype, n, c, with_res):
    x, w = _rand(n, n, c, dtype=dtype), _rand(c, c, dtype=dtype)
    res = _rand(n + 1, n, c, dtype=dtype, scale=3.0) if with_res else None
    r = scv.rms_norm_fwd(x, w, res, 1e-5, q8=True, q8_h=True)
    h, rstd, y = plain_norm(x, res, w, float(np.float32(1e-5)))
    u, tiny = UNIT[dtype], TINY[dtype]
    _within(r.rstd, rstd, OWN * rstd, "rstd")
    _within(r.y, y, (u + OWN) * y.abs() + tiny, "y")
    if with_res:
        _within(r.h, h, (u + 2.0 ** -24) * h.abs() + tiny, "h")
    else:
        assert r.h is x
    _check_q8(r.y8, y, OWN, "y in 8 bits")
    _check_q8(r.h8, h, 2.0 ** -24, "h in 8 bits")


def test_norm_outputs_alone_and_in_place():
    """Each output on its own equals the one of the full call; h over x or over res."""
    x, res, w = (_rand(i, 300, 136, dtype=torch.bfloat16) for i in range(3))
    w = w[0].contiguous()
    full = scv.rms_norm_fwd(x, w, res, q8=True, q8_h=True)
    only = scv.rms_norm_fwd(x, w, res, rows=False, q8=True)
    assert only.y is None and only.h8 is None
    assert torch.equal(only.y8.q.view(torch.uint8), full.y8.q.view(torch.uint8))
    assert torch.equal(only.y8.scale, full.y8.scale)
    for over in (0, 1):
        a = [x.clone(), res.clone()]
        r = scv.rms_norm_fwd(a[0], w, a[1], h_out=a[over])
        assert r.h is a[over] and torch.equal(r.h, full.h) and torch.equal(r.y, full.y)
    ones = scv.rms_norm_fwd(x, None, res)
    assert torch.equal(ones.y, scv.rms_norm_fwd(x, torch.ones_like(w), res).y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_special_rows(dtype):
    """A row of zeros gives zeros, tiny rows what eps leaves of them, a NaN or an infinity stays in its own row."""
    x = _rand(5, 6, 64, dtype=dtype)
    x[1] = 0
    x[2] = 1e-4
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    w = _rand(6, 64, dtype=dtype)
    r = scv.rms_norm_fwd(x, w, q8=True)
    assert not r.y[1].any() and not values_q8(r.y8)[1].any()
    clean = [0, 1, 2, 5]
    _, _, y = plain_norm(x[clean], None, w, float(np.float32(1e-6)))
    _within(r.y[clean], y, (UNIT[dtype] + OWN) * y.abs() + TINY[dtype], "y")
    assert bool(torch.isnan(r.y[3]).all()) and bool(torch.isnan(r.y8.q[3].float()).all())
    assert bool(torch.isfinite(r.y[clean]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,c", [(3, 64), (2, 16384)])
def test_norm_of_the_largest_rows(dtype, n, c):
    """Magnitudes up to 10^17, whose squares' sum ends below fp32's largest number at any channel count, both ways."""
    x, w, dy = (1e17 * (2 * torch.rand(n, c, generator=torch.Generator().manual_seed(c)) - 1)).to(dtype).cuda(), \
        _rand(c, c, dtype=dtype), _rand(n, n, c, dtype=dtype)
    x[0] = 9.9e16
    r = scv.rms_norm_fwd(x, w, q8=True, q8_h=True)
    h, rstd, y = plain_norm(x, None, w, float(np.float32(1e-6)))
    _within(r.rstd, rstd, OWN * rstd, "rstd")
    _within(r.y, y, (UNIT[dtype] + OWN) * y.abs() + TINY[dtype], "y")
    _check_q8(r.h8, h, 2.0 ** -24, "h in 8 bits")
    for saved, plain in ((r.h, h), (r.h8, values_q8(r.h8))):
        dx, dw = scv.rms_norm_bwd(dy, saved, r.rstd, w)
        ref, own, dw_ref, mag = plain_norm_bwd(dy, plain, r.rstd, w, None)
        _within(dx, ref, UNIT[dtype] * (ref.abs() + own) + own + TINY[dtype], "dx")
        _within(dw, dw_ref, 128 * 2.0 ** -24 * mag, "dw")


def plain_norm_bwd(dy, h, rstd, w, dh):
    """dx, its bound without the output's rounding, dw and the magnitudes of its terms, in 64 bits."""
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    xh = h * r
    g = dy if w is None else dy * w.double()
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    own = 2.0 ** -17 * r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        own = own + 2.0 ** -23 * dh.double().abs()
    return dx, own, (dy * xh).sum(0), (dy * xh).abs().sum(0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", SHAPES + [(20000, 64), (0, 64)])
@pytest.mark.parametrize("saved", ["rows", "8bit"])
def test_norm_gradient(dtype, n, c, saved):
    x, dy, dh = (_rand(n + i, n, c, dtype=dtype) for i in range(3))
    w = _rand(c, c, dtype=dtype) if c != 264 else None
    dh = None if c in (16, 512) else dh
    f = scv.rms_norm_fwd(x, w, q8_h=True)
    h = f.h if saved == "rows" else f.h8
    dx, dw = scv.rms_norm_bwd(dy, h, f.rstd, w, dh)
    ref, own, dw_ref, mag = plain_norm_bwd(dy, f.h if saved == "rows" else values_q8(f.h8), f.rstd, w, dh)
    _within(dx, ref, UNIT[dtype] * (ref.abs() + own) + own + TINY[dtype], "dx")
    # a share's sum, its groups', then the shares': at most n / 592 + 64 + 19 + 32 additions deep, and the product's roundings
    _within(dw, dw_ref, (n / 592 + 128) * 2.0 ** -24 * mag, "dw")
    again, dw2 = scv.rms_norm_bwd(dy, h, f.rstd, w, dh)
    assert torch.equal(dx, again) and torch.equal(dw, dw2), "the bits depend on timing"
    assert scv.rms_norm_bwd(dy, h, f.rstd, w, dh, want_dw=False)[1] is None
    for over in ([dy] if dh is None else [dy, dh]):  # dx in place of dy or dh
        a = over.clone()
        got, _ = scv.rms_norm_bwd(a if over is dy else dy, h, f.rstd, w, a if over is dh else dh, out=a)
        assert got is a and torch.equal(a, dx)


def test_norm_gradients_from_two_host_threads():
    """One thread's rows have another gradient added, which takes more shared memory of the same kernel; none of the
    calls fails."""
    rows = [[_rand(i, 8, 8192, dtype=torch.bfloat16) for i in range(k, k + 3)] for k in (0, 10)]
    f = [scv.rms_norm_fwd(r[0]) for r in rows]
    want = [scv.rms_norm_bwd(r[1], x.h, x.rstd, dh=d)[0] for r, x, d in zip(rows, f, (None, rows[1][2]))]
    torch.cuda.synchronize()
    wrong = []

    def calls(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(400):
                    dx, _ = scv.rms_norm_bwd(rows[k][1], f[k].h, f[k].rstd, dh=rows[1][2] if k else None, want_dw=False)
                torch.cuda.current_stream().synchronize()
            if not torch.equal(dx, want[k]):
                wrong.append("another result")
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=calls, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_norm_gradient_against_differences():
    """Central differences of L = sum(y a) + sum(h b), in 64 bits with step d: their own error is at most
    d^2 times the third derivative, far below the fp32 bound used here."""
    n, c, d = 6, 24, 2.0 ** -10
    x, res, a, b = (_rand(20 + i, n, c) for i in range(4))
    w = _rand(30, c)
    f = scv.rms_norm_fwd(x, w, res)
    dx, dw = scv.rms_norm_bwd(a, f.h, f.rstd, w, b)

    def loss(xx, ww):
        h, _, y = plain_norm(xx, res, ww, 1e-6)
        return (y * a.double()).sum() + (h * b.double()).sum()

    for i, j in [(0, 0), (2, 5), (5, 23), (3, 11)]:
        e = torch.zeros(n, c, dtype=torch.float64, device="cuda")
        e[i, j] = d
        num = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * d)
        assert abs(float(num) - float(dx[i, j])) <= 2e-5 * (1 + abs(float(num)))
        e = torch.zeros(c, dtype=torch.float64, device="cuda")
        e[j] = d
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * d)
        assert abs(float(num) - float(dw[j])) <= 2e-5 * (1 + abs(float(num)))


# --------------------------------------------------------------------------- weight gradient from 8-bit rows
def _subm(coords):
    c = torch.from_numpy(coords).cuda()
    st = scv.new_status()
    km = scv.kernel_map(scv.hash_table(c, 4.0, st), len(coords), c, scv.subm_geom(3), d_status=st)
    scv.check_status(st)
    return km, oracle.kmap(coords, coords, 3, 1, 1, oracle.SUBM)


@pytest.mark.parametrize("n", [1, 40, 3000])
@pytest.mark.parametrize("cin,cout,dtype", [
    (8, 32, torch.float32), (16, 16, torch.float32), (40, 72, torch.float32), (24, 16, torch.bfloat16),
    (64, 64, torch.float16), (64, 128, torch.bfloat16), (128, 64, torch.float16), (128, 128, torch.bfloat16),
    (128, 128, torch.float16), (64, 64, torch.bfloat16), (64, 64, torch.float32), (256, 8, torch.float16),
])
def test_weight_gradient_from_8bit_rows(n, cin, cout, dtype):
    """The products are exact in fp32 and each addition is off by at most one step (the tensor cores cut off)."""
    coords = rand_coords(np.random.default_rng(n + cin), n, -9, 9)
    km, nbr = _subm(coords)
    r = scv.q8_pack(_rand(cin, n, cin, dtype=dtype))
    dy = _rand(cout, n, cout, dtype=dtype)
    st = scv.new_status()
    dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
    scv.check_status(st)
    x64, g64 = values_q8(r).cpu().numpy(), dy.double().cpu().numpy()
    ref = oracle.conv_wgrad(x64, g64, nbr)
    mag = oracle.conv_wgrad(np.abs(x64), np.abs(g64), nbr)
    terms = (nbr >= 0).sum(0)[:, None, None] + 64
    err = np.abs(dw.double().cpu().numpy() - ref)
    assert np.all(err <= terms * 2.0 ** -23 * mag), float((err / np.maximum(mag, 1e-300)).max())
    assert torch.equal(dw, scv.conv_wgrad_q8(r, dy, km)), "the bits depend on timing"


@pytest.mark.parametrize("level", ["low", "high"])
@pytest.mark.parametrize("packed", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cin,cout", [(16, 16), (40, 24), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_weight_gradient_in_fp16_takes_the_rows_as_fp16(cin, cout, packed, level):
    """Rows from a type of another range: groups whose values lie below fp16's normal numbers (and partly below all of
    them), or above its largest.  Whatever the channel counts, x is what q8_unpack writes in fp16."""
    coords = rand_coords(np.random.default_rng(cin + cout), 3000, -8, 8)
    km, nbr = _subm(coords)
    n, group = len(coords), torch.arange(cin) // 32
    power = torch.where(group % 2 == 0, -20, -26) if level == "low" else torch.where(group % 2 == 0, 17, 13)
    r = scv.q8_pack((_rand(cin, n, cin) * (2.0 ** power).cuda()).to(packed))
    e = r.scale.int()
    assert bool((e < 112).all() if level == "low" else (e[:, 0] > 134).all())
    x = values_q8(r).clamp(-65504.0, 65504.0).to(torch.float16)
    assert not torch.equal(x.double(), values_q8(r)) and torch.equal(x, scv.q8_unpack(r, torch.float16))
    dy = _rand(cout, n, cout, dtype=torch.float16)
    st = scv.new_status()
    dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
    scv.check_status(st)
    x, g = x.double(), dy.double()
    for k in range(27):
        j = np.nonzero(nbr[:, k] >= 0)[0]
        i, j = torch.from_numpy(nbr[j, k].astype(np.int64)).cuda(), torch.from_numpy(j).cuda()
        ref, mag = x[i].t() @ g[j], x[i].abs().t() @ g[j].abs()
        _within(dw[k], ref, (len(j) + 64) * 2.0 ** -23 * mag, f"offset {k}")


@pytest.mark.parametrize("cin,cout,dtype", [(64, 64, torch.bfloat16), (128, 64, torch.float16)])
def test_weight_gradient_of_long_shares(cin, cout, dtype):
    """A million pairs: shares of several thousand pairs of one offset, whose sums leave the accumulator more than once."""
    coords = rand_coords(np.random.default_rng(5), 40000, -18, 18)
    km, nbr = _subm(coords)
    r = scv.q8_pack(_rand(1, len(coords), cin, dtype=dtype))
    dy = _rand(2, len(coords), cout, dtype=dtype)
    dw = scv.conv_wgrad_q8(r, dy, km)
    x, g = values_q8(r), dy.double()
    for k in (0, 13, 20, 26):
        j = np.nonzero(nbr[:, k] >= 0)[0]
        i, j = torch.from_numpy(nbr[j, k].astype(np.int64)).cuda(), torch.from_numpy(j).cuda()
        ref, mag = x[i].t() @ g[j], x[i].abs().t() @ g[j].abs()
        _within(dw[k], ref, (2048 + 64) * 2.0 ** -23 * mag, f"offset {k}")


@pytest.mark.parametrize("cin,cout,dtype", [(64, 64, torch.float16), (128, 128, torch.bfloat16), (64, 128, torch.bfloat16),
                                            (128, 64, torch.float16)])
def test_weight_gradient_of_sums_longer_than_an_accumulator_takes(cin, cout, dtype):
    """A full cube of 48^3 voxels: 2.9 million pairs in 592 shares, each longer than the 64 blocks of 64 pairs after which
    two groups' accumulators are emptied into the segment's total, so that most segments empty them twice.  With values of
    one sign a part that was lost or added twice would be some hundredths of the sum, the bound is 2.5e-4 of it."""
    side = 48
    coords = np.stack(np.meshgrid(np.zeros(1), *[np.arange(side)] * 3, indexing="ij"), -1).reshape(-1, 4).astype(np.int32)
    coords = np.ascontiguousarray(coords[np.random.default_rng(12).permutation(len(coords))])
    km, nbr = _subm(coords)
    pairs = int((nbr >= 0).sum())
    assert pairs == (3 * side - 2) ** 3 and pairs // (4 * 148) > 64 * 64
    n = len(coords)
    for sign in (False, True):
        x, g = _rand(1, n, cin, dtype=dtype), _rand(2, n, cout, dtype=dtype)
        r, dy = scv.q8_pack(x.abs() if sign else x), g.abs() if sign else g
        st = scv.new_status()
        dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
        scv.check_status(st)
        x, g = values_q8(r), dy.double()
        for k in range(27):
            j = np.nonzero(nbr[:, k] >= 0)[0]
            i, j = torch.from_numpy(nbr[j, k].astype(np.int64)).cuda(), torch.from_numpy(j).cuda()
            ref, mag = x[i].t() @ g[j], x[i].abs().t() @ g[j].abs()
            _within(dw[k], ref, (2048 + 64) * 2.0 ** -23 * mag, f"offset {k}")
        assert torch.equal(dw, scv.conv_wgrad_q8(r, dy, km)), "the bits depend on timing"


@pytest.mark.parametrize("n", [64, 65, 4999, 30011])
@pytest.mark.parametrize("cin,cout,dtype", [(64, 128, torch.bfloat16), (128, 64, torch.float16)])
def test_weight_gradient_of_a_map_that_is_mostly_centre(n, cin, cout, dtype):
    """Voxels with hardly a neighbour: blocks of consecutive rows, and an offset that every worker has several shares of."""
    coords = rand_coords(np.random.default_rng(n), n, -120, 120)
    km, nbr = _subm(coords)
    r = scv.q8_pack(_rand(n, n, cin, dtype=dtype))
    dy = _rand(n + 1, n, cout, dtype=dtype)
    st = scv.new_status()
    dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
    scv.check_status(st)
    x, g = values_q8(r), dy.double()
    for k in range(27):
        j = np.nonzero(nbr[:, k] >= 0)[0]
        i, j = torch.from_numpy(nbr[j, k].astype(np.int64)).cuda(), torch.from_numpy(j).cuda()
        ref, mag = x[i].t() @ g[j], x[i].abs().t() @ g[j].abs()
        _within(dw[k], ref, (len(j) + 64) * 2.0 ** -23 * mag, f"offset {k}")
    # scales from an address that is not a multiple of 16: gathered instead
    odd = torch.empty(r.scale.numel() + 4, dtype=torch.uint8, device="cuda")[4:].view(r.scale.shape)
    odd.copy_(r.scale)
    assert torch.equal(scv.conv_wgrad_q8(scv.Q8Rows(r.q, odd), dy, km), dw)


@pytest.mark.parametrize("cin,cout,dtype", [(64, 64, torch.bfloat16), (64, 128, torch.float16), (128, 64, torch.bfloat16)])
def test_weight_gradient_of_rows_with_scales_of_their_own(cin, cout, dtype):
    """Neighbouring rows, and neighbouring groups of a row, whose scales are powers of two apart: a pair that took
    another one's scale byte would be off by its factor.  Called many times, the bits stay."""
    coords = rand_coords(np.random.default_rng(11), 9001, -12, 12)
    km, nbr = _subm(coords)
    n = len(coords)
    factor = 2.0 ** ((torch.arange(n)[:, None] * 5 + torch.arange(cin) // 32 * 3) % 13 - 6).cuda()
    r = scv.q8_pack((_rand(3, n, cin) * factor).to(dtype))
    dy = _rand(4, n, cout, dtype=dtype)
    st = scv.new_status()
    dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
    scv.check_status(st)
    x, g = values_q8(r), dy.double()
    for k in range(27):
        j = np.nonzero(nbr[:, k] >= 0)[0]
        i, j = torch.from_numpy(nbr[j, k].astype(np.int64)).cuda(), torch.from_numpy(j).cuda()
        ref, mag = x[i].t() @ g[j], x[i].abs().t() @ g[j].abs()
        _within(dw[k], ref, (2048 + 64) * 2.0 ** -23 * mag, f"offset {k}")
    ws = scv.Workspace()
    for _ in range(50):
        assert torch.equal(dw, scv.conv_wgrad_q8(r, dy, km, ws))


def test_weight_gradient_wait_that_runs_out():
    """With no time to wait the kernel gives up, says so and leaves the GPU in order: the next call is right."""
    coords = rand_coords(np.random.default_rng(6), 5000, -12, 12)
    km, _ = _subm(coords)
    r, dy = scv.q8_pack(_rand(1, 5000, 64, dtype=torch.bfloat16)), _rand(2, 5000, 64, dtype=torch.bfloat16)
    want = scv.conv_wgrad_q8(r, dy, km)
    st = scv.new_status()
    was = scv.lat_set_wait_limit_ns(0)
    try:
        scv.conv_wgrad_q8(r, dy, km, d_status=st)
        torch.cuda.synchronize()
    finally:
        scv.lat_set_wait_limit_ns(was)
    with pytest.raises(scv.LatticeError, match="LAT_ERR_TIMEOUT"):
        scv.check_status(st)
    assert torch.equal(scv.conv_wgrad_q8(r, dy, km), want)


def test_weight_gradient_flags_a_bad_pair():
    """A row index outside the rows is flagged and its pair left out (the map is checked before the rows are read)."""
    coords = rand_coords(np.random.default_rng(7), 500, -5, 5)
    km, _ = _subm(coords)
    for c, dtype in ((64, torch.bfloat16), (16, torch.float32)):
        r, dy = scv.q8_pack(_rand(1, 500, c, dtype=dtype)), _rand(2, 500, c, dtype=dtype)
        kept = km.pair_in[3].clone()
        km.pair_in[3] = 500
        st = scv.new_status()
        dw = scv.conv_wgrad_q8(r, dy, km, d_status=st)
        with pytest.raises(scv.LatticeError, match="LAT_ERR_BAD_MAP"):
            scv.check_status(st)
        assert bool(torch.isfinite(dw).all())
        km.pair_in[3] = kept


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient_from_8bit_rows_of_a_strided_map(dtype):
    """n_in and n_out differ: the coarse rows of a k=2, stride-2 convolution."""
    coords = rand_coords(np.random.default_rng(8), 2500, -9, 9, 2)
    c = torch.from_numpy(coords).cuda()
    g = scv.strided_geom(2, 2, 0)
    coarse = scv.downsample(c, g).contiguous()
    km = scv.kernel_map(scv.hash_table(c), len(coords), coarse, g)
    nbr = oracle.kmap(coords, coarse.cpu().numpy(), 2, 2, 0, oracle.STRIDED)
    r = scv.q8_pack(_rand(1, len(coords), 64, dtype=dtype))
    dy = _rand(2, len(coarse), 128, dtype=dtype)
    dw = scv.conv_wgrad_q8(r, dy, km)
    x64, g64 = values_q8(r).cpu().numpy(), dy.double().cpu().numpy()
    err = np.abs(dw.double().cpu().numpy() - oracle.conv_wgrad(x64, g64, nbr))
    mag = oracle.conv_wgrad(np.abs(x64), np.abs(g64), nbr)
    assert np.all(err <= ((nbr >= 0).sum(0)[:, None, None] + 64) * 2.0 ** -23 * mag)


def test_weight_gradient_of_a_map_without_rows():
    km = scv.KernelMap(0, 0, 27)
    km.pair_off.zero_()
    r = scv.Q8Rows.empty(0, 64)
    assert not scv.conv_wgrad_q8(r, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), km).any()


# --------------------------------------------------------------------------- together
class Step:
    """One residual block in a training step: rows from token ids, norm, convolution, and back, with 8-bit checkpoints."""

    def __init__(self, dtype=torch.bfloat16, c=64, vocab=50):
        self.coords = rand_coords(np.random.default_rng(77), 1500, -8, 8)
        self.n, self.c, self.vocab, self.dtype = len(self.coords), c, vocab, dtype
        self.km, self.nbr = _subm(self.coords)
        self.table, self.g = _rand(1, vocab, c, dtype=dtype), _rand(2, c, dtype=dtype)
        self.w = _rand(3, 27, c, c, dtype=dtype, scale=(27 * c) ** -0.5)
        self.ids, self.res = _ids(4, self.n, vocab, torch.int32), _rand(5, self.n, c, dtype=dtype)
        self.dy, self.dh = _rand(6, self.n, c, dtype=dtype), _rand(7, self.n, c, dtype=dtype)
        self.ws = scv.Workspace()

    def run(self, stream=None):
        k = dict(stream=stream)
        x = scv.embed_fwd(self.ids, self.table, 2.0, **k)
        f = scv.rms_norm_fwd(x, self.g, self.res, q8=True, q8_h=True, **k)
        y = scv.conv_fwd(f.y, self.w, self.km, self.ws, **k)
        dw = scv.conv_wgrad_q8(f.y8, self.dy, self.km, self.ws, **k)
        dn = scv.conv_dgrad(self.dy, self.w, self.km, True, self.ws, **k)
        dx, dg = scv.rms_norm_bwd(dn, f.h8, f.rstd, self.g, self.dh, ws=self.ws, **k)
        dt = scv.embed_wgrad(self.ids, dx, self.vocab, 2.0, ws=self.ws, **k)
        return [x, f.h, f.rstd, f.y, f.y8.q.view(torch.uint8), f.y8.scale, y, dw, dn, dx, dg, dt]


def test_a_step_of_them_together():
    """Each operator of the chain against its own formula, on the inputs that the chain gave it."""
    s = Step()
    x, h, rstd, y, y8, y8s, out, dw, dn, dx, dg, dt = s.run()
    have = (s.ids >= 0)[:, None]
    assert torch.equal(x, torch.where(have, s.table[s.ids.long().clamp(min=0)] * 2, 0))
    _, _, yr = plain_norm(x, s.res, s.g, float(np.float32(1e-6)))
    _within(y, yr, (UNIT[s.dtype] + OWN) * yr.abs() + TINY[s.dtype], "y")
    x64 = values_q8(scv.Q8Rows(y8.view(torch.float8_e4m3fn), y8s)).cpu().numpy()
    g64 = s.dy.double().cpu().numpy()
    err = np.abs(dw.double().cpu().numpy() - oracle.conv_wgrad(x64, g64, s.nbr))
    assert np.all(err <= 1600 * 2.0 ** -23 * oracle.conv_wgrad(np.abs(x64), np.abs(g64), s.nbr))
    h8 = scv.q8_pack((x.float() + s.res.float()))
    ref, own, dg_ref, mag = plain_norm_bwd(dn, values_q8(h8), rstd, s.g, s.dh)
    _within(dx, ref, UNIT[s.dtype] * (ref.abs() + own) + own + TINY[s.dtype], "dx")
    _within(dg, dg_ref, 256 * 2.0 ** -24 * mag, "dg")
    at = s.ids.long() % (s.vocab + 1)
    zero = torch.zeros(s.vocab + 1, s.c, dtype=torch.float64, device="cuda")
    ref, mag = zero.index_add(0, at, dx.double())[:-1] * 2, zero.index_add(0, at, dx.double().abs())[:-1] * 2
    _within(dt, ref, 1500 * 2.0 ** -24 * mag, "dtable")


def test_a_step_on_another_stream_and_captured():
    """The same bits on a side stream, by its raw handle, and from a captured graph replayed on new inputs while another
    graph of the same step, with the workspace in common, is replayed in between."""
    s = Step()
    want = s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = s.run(stream)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = s.run()
        graphs.append((g, outs))
    s.ids.copy_(_ids(9, s.n, s.vocab, torch.int32))
    s.dy.copy_(_rand(10, s.n, s.c, dtype=s.dtype))
    s.res.mul_(0.5)
    for g, _ in graphs + graphs[:1]:
        g.replay()
    torch.cuda.synchronize()
    want = s.run()
    for _, outs in graphs:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_lookup_gradient_of_a_large_table_captured():
    """Zeros of many megabytes take the side stream, inside a capture too, and in a thread whose first call is captured."""
    ids, dy = _ids(3, 9000, 40000, torch.int64), _rand(4, 9000, 128, dtype=torch.bfloat16)
    want = scv.embed_wgrad(ids, dy, 40000)
    ws = scv.Workspace()
    out = scv.embed_wgrad(ids, dy, 40000, ws=ws).fill_(float("nan"))

    def captured(got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            scv.embed_wgrad(ids, dy, 40000, ws=ws, out=out)
        for _ in range(2):
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            got.append(out.clone())

    got = []
    captured(got)
    thread = threading.Thread(target=captured, args=(got,))
    thread.start()
    thread.join()
    assert len(got) == 4 and all(torch.equal(o, want) for o in got)


def test_lookup_gradients_in_one_capture():
    """Two of them in a row share the side stream and the workspace."""
    ids = [_ids(i, n, 40000, torch.int64) for i, n in enumerate((9000, 300))]
    dy = [_rand(i, n, 128) for i, n in enumerate((9000, 300))]
    want = [scv.embed_wgrad(i, d, 40000) for i, d in zip(ids, dy)]
    ws = scv.Workspace()
    out = [scv.embed_wgrad(i, d, 40000, ws=ws).fill_(float("nan")) for i, d in zip(ids, dy)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, d, o in zip(ids, dy, out):
            scv.embed_wgrad(i, d, 40000, ws=ws, out=o)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_two_streams_at_once():
    """Calls with their own workspaces on two streams do not disturb one another."""
    ids = [_ids(i, 60000, 500, torch.int64) for i in range(2)]
    dy = [_rand(i, 60000, 64, dtype=torch.bfloat16) for i in range(2)]
    want = [scv.embed_wgrad(i, d, 500) for i, d in zip(ids, dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for k in range(2):
            got[k].append(scv.embed_wgrad(ids[k], dy[k], 500, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(g, want[k]) for g in got[k])


@pytest.mark.parametrize("in_threads", [False, True])
def test_gradients_of_large_tables_on_two_streams_at_once(in_threads):
    """From one host thread they share its side stream, from two each has its own; outputs of a call that follows on
    the same stream are not overwritten by zeros that are still on their way."""
    vocab = 40000
    ids = [_ids(20 + i, n, vocab, torch.int64) for i, n in enumerate((9000, 30000))]
    dy = [_rand(20 + i, len(d), 128, dtype=torch.bfloat16) for i, d in enumerate(ids)]
    want = [scv.embed_wgrad(i, d, vocab) for i, d in zip(ids, dy)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    same = [[], []]

    def calls(k):
        with torch.cuda.stream(streams[k]):
            ws, out = scv.Workspace(), torch.empty(vocab, 128, device="cuda")
            for _ in range(6):
                scv.embed_wgrad(ids[k], dy[k], vocab, ws=ws, out=out.fill_(float("nan")))
                same[k].append((out == want[k]).all())
            streams[k].synchronize()

    if in_threads:
        threads = [threading.Thread(target=calls, args=(k,)) for k in (0, 1)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    else:
        for k in (0, 1, 0):
            calls(k)
        ws, out = [scv.Workspace() for _ in range(2)], [torch.empty(vocab, 128, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(6):
            for k in (0, 1):
                scv.embed_wgrad(ids[k], dy[k], vocab, ws=ws[k], out=out[k], stream=streams[k])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(out, want))
    assert all(len(v) >= 6 and all(v) for v in same)


def test_rows_past_32_bit_offsets():
    """More than 2^31 values: the last rows come out as on their own."""
    n, c = (1 << 31) // 8192 + 40, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, c, generator=g, device="cuda", dtype=torch.bfloat16)
    w = _rand(1, c, dtype=torch.bfloat16)
    f = scv.rms_norm_fwd(x, w, q8=True, q8_h=True)
    last = scv.rms_norm_fwd(x[-50:].contiguous(), w, q8=True)
    assert torch.equal(f.y[-50:], last.y) and torch.equal(f.y8.scale[-50:], last.y8.scale)
    assert torch.equal(f.y8.q[-50:].view(torch.uint8), last.y8.q.view(torch.uint8))
    assert torch.equal(scv.q8_unpack(f.y8)[-50:], scv.q8_unpack(last.y8))
    dx, _ = scv.rms_norm_bwd(x, f.h8, f.rstd, w, want_dw=False)
    alone = scv.q8_pack(x[-50:].contiguous())
    assert torch.equal(dx[-50:], scv.rms_norm_bwd(x[-50:].contiguous(), alone, f.rstd[-50:].contiguous(), w)[0])
    del f, dx
    ids = torch.arange(n - 50, n, device="cuda", dtype=torch.int32)
    assert torch.equal(scv.embed_fwd(ids, x), x[-50:])
    rows = torch.full((n,), -1, device="cuda", dtype=torch.int32)
    rows[-50:] = torch.arange(50, dtype=torch.int32)
    assert torch.equal(scv.embed_wgrad(rows, x, 50), x[-50:].float())


def test_a_gradient_past_32_bit_offsets():
    """A table of more than 2^31 values: tokens at both ends, and zeros in all the rows between."""
    vocab, c = (1 << 31) // 8192 + 40, 8192
    ids = torch.tensor([vocab - 1, 3, vocab - 1, vocab - 40, 0, 3], dtype=torch.int32, device="cuda")
    dy = _rand(9, 6, c, dtype=torch.bfloat16)
    for rows in (1, 1000):    # sorted by one block, and by launches with the zeros beside them
        out = torch.full((vocab, c), float("nan"), device="cuda")
        dt = scv.embed_wgrad(ids.repeat(rows), dy.repeat(rows, 1), vocab, out=out)
        have = torch.unique(ids).long()
        slot = torch.searchsorted(have, ids.long())
        ref, mag = (torch.zeros(len(have), c, dtype=torch.float64, device="cuda").index_add_(0, slot, rows * d)
                    for d in (dy.double(), dy.double().abs()))
        _within(dt[have], ref, (2 * rows + 2) * 2.0 ** -24 * mag, "gradient")
        dt[have] = 0
        assert not dt.any()
        del out, dt


def test_calls_without_rows():
    """Nothing to do, and a gradient of zeros: no call refuses it."""
    table, st = _rand(1, 20, 64, dtype=torch.bfloat16), scv.new_status()
    none = table[:0]
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    assert scv.embed_fwd(ids, table, d_status=st).shape == (0, 64)
    assert not scv.embed_wgrad(ids, none, 20, d_status=st).any()
    f = scv.rms_norm_fwd(none, table[0].contiguous(), none.clone(), q8=True, q8_h=True)
    assert f.y.shape == f.h.shape == f.y8.shape == f.h8.shape == (0, 64) and f.rstd.shape == (0,)
    for h in (f.h, f.h8):
        dx, dw = scv.rms_norm_bwd(none, h, f.rstd, table[0].contiguous())
        assert dx.shape == (0, 64) and not dw.any()
    assert scv.q8_unpack(scv.q8_pack(none)).shape == (0, 64)
    scv.check_status(st)


def test_refusal_of_tensors_that_are_not_contiguous():
    x = _rand(1, 8, 64)
    with pytest.raises(ValueError, match="contiguous"):
        scv.rms_norm_fwd(x[:, :32])
    with pytest.raises(ValueError, match="contiguous"):
        scv.q8_pack(x.t())
    with pytest.raises(scv.LatticeError, match="LAT_ERR_ARG"):
        scv.q8_pack(x.flatten()[2:2 + 64].view(1, 64))   # 8 bytes off a 16-byte boundary
