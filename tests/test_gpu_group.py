"""GPU parity of the expert-grouped path (dispatch, products, gradients,
combine) against the fp64 oracle.

Tolerances, per element, on the same 16-bit inputs:
  a product's fp32 sum of T exact products: T * 2^-24 * sum|a b| (one half-step
  per addition, in any order), plus the output's rounding, half a step
  (torch.finfo(type).eps / 2) of the value, plus half the smallest subnormal;
  silu: 1 / (1 + e^-g) through a hardware exponential of -g log2(e) rounded to
  fp32 (relative (|g| + 4) * 2^-22), and the products' errors carried through
  |d silu / dg| <= 1.1, |d2| <= 0.6.
Tiles are 64 to 256 wide, so the sizes below end inside one, at one, past one."""

import numpy as np
import pytest

from oracle import group as OG

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from bit_moe_expert_02_amd import _lib as L          # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _half_step(ref, dtype):
    eps = torch.finfo(dtype).eps
    return np.abs(ref) * eps / 2 + torch.finfo(dtype).smallest_normal * eps / 2


def _close(got, ref, tol, what=""):
    got = _f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol):.3g} tolerances, " \
        f"first at {np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {ref[bad][0]}"


class Case:
    """Ragged rows, an operand (gathered or not), weights; every array inside a larger one of sentinels when
    `pad` (row strides past the width, a start off 16 bytes)."""

    def __init__(self, counts, n, k, dtype, x_cols, gather=False, pad=0, first=0, tail=3, seed=0):
        rng = np.random.default_rng(seed + 7 * n + k)
        self.counts, self.n, self.k, self.dtype, self.pad = counts, n, k, dtype, pad
        self.groups = len(counts)
        self.offsets_h = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.offsets_h[-1]) + tail
        self.div = 2 if gather else 1
        x_rows = max(1, self.rows // 2 + 2) if gather else self.rows
        self.x = self.matrix(rng.standard_normal((x_rows, x_cols)), dtype)
        self.w = self.matrix(rng.standard_normal((self.groups * n, k)) * 0.1, dtype, groups=self.groups)
        self.src = self.src_h = None
        if gather:
            self.src_h = rng.integers(0, 2 * x_rows, self.rows).astype(np.int32)
            self.src_h[::5] = -1                        # rows of zeros
            self.src_h[1::7] = 2 * x_rows
            self.src = _dev(self.src_h, torch.int32)
        self.offsets = _dev(self.offsets_h, torch.int32)
        self.xg = OG.gathered(_f64(self.x), self.src_h, self.div)
        if not gather:
            self.xg = _f64(self.x)
        self.wf = _f64(self.w)

    def matrix(self, a, dtype, groups=None):
        """A device tensor of a; with pad, a view into a larger buffer."""
        r, c = a.shape
        if not self.pad:
            t = _dev(a, dtype)
            return t if groups is None else t.view(groups, r // groups, c)
        if groups is None:
            buf = torch.full((r * (c + self.pad) + 1,), SENTINEL, dtype=dtype, device="cuda")
            t = buf[1:].view(r, c + self.pad)[:, :c]
        else:
            n = r // groups
            buf = torch.full((groups * (n + 1) * (c + self.pad) + 1,), SENTINEL, dtype=dtype, device="cuda")
            t = buf[1:].view(groups, n + 1, c + self.pad)[:, :n, :c]
        t.copy_(_dev(a, dtype).view(t.shape))
        return t

    def out(self, cols, dtype):
        """(whole buffer, the view a call writes)."""
        whole = torch.full((self.rows, cols + self.pad), SENTINEL, dtype=dtype, device="cuda")
        return whole, whole[:, :cols]

    def held(self):
        m = np.zeros(self.rows, bool)
        m[self.offsets_h[0]:self.offsets_h[-1]] = True
        return m

    def check(self, whole, view, ref, tol, what):
        torch.cuda.synchronize()
        m = self.held()
        _close(view[torch.from_numpy(m).cuda()], ref[m], tol[m], what)
        rest = whole.clone()
        rest[self.offsets_h[0]:self.offsets_h[-1], :view.shape[1]] = SENTINEL
        assert bool((rest == SENTINEL).all()), f"{what}: wrote outside its rows or columns"


def _sum_tol(xa, wa, terms, offsets, rows, fn):
    return (terms + 2) * 2.0**-24 * fn(np.abs(xa), offsets, np.abs(wa), rows)


RAGGED = [3, 0, 1, 64, 0, 130, 7]
MANY = [300, 1, 513, 40, 260]
SHAPES = [(RAGGED, 64, 64), (RAGGED, 1, 1), (RAGGED, 17, 33), (RAGGED, 130, 257), ([1], 256, 512), (RAGGED, 515, 261),
          ([200], 96, 8), (MANY, 768, 832), (MANY, 512, 72), ([70] * 70, 72, 64), ([0, 0], 64, 64), (MANY, 300, 456)]
VARIANTS = [dict(), dict(gather=True), dict(pad=3), dict(pad=8, first=5), dict(gather=True, pad=1)]


@pytest.mark.parametrize("variant", range(len(VARIANTS)))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matmul_and_its_input_gradient(shape, dtype, out, variant):
    counts, n, k = SHAPES[shape]
    c = Case(counts, n, k, dtype, k, seed=shape, **VARIANTS[variant])
    whole, y = c.out(n, out)
    L.moe_group_matmul(c.x, c.offsets, c.w, y, src=c.src, src_div=c.div)
    ref = OG.matmul(c.xg, c.offsets_h, c.wf, c.rows)
    c.check(whole, y, ref, _sum_tol(c.xg, c.wf, k, c.offsets_h, c.rows, OG.matmul) + _half_step(ref, out), "matmul")

    c = Case(counts, n, k, dtype, n, seed=shape + 50, **VARIANTS[variant])
    whole, dx = c.out(k, out)
    L.moe_group_matmul_t(c.x, c.offsets, c.w, dx, src=c.src, src_div=c.div)
    ref = OG.matmul_t(c.xg, c.offsets_h, c.wf, c.rows)
    c.check(whole, dx, ref, _sum_tol(c.xg, c.wf, n, c.offsets_h, c.rows, OG.matmul_t) + _half_step(ref, out), "matmul_t")


def _silu_rel(g):
    return (np.abs(g) + 4) * 2.0**-22


@pytest.mark.parametrize("variant", range(len(VARIANTS)))
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("counts,half,k", [(RAGGED, 32, 64), (RAGGED, 1, 5), (RAGGED, 33, 129), (MANY, 300, 264), (MANY, 384, 512)])
def test_swiglu_and_its_gradient(counts, half, k, dtype, out, variant):
    c = Case(counts, 2 * half, k, dtype, k, seed=half, **VARIANTS[variant])
    whole, h = c.out(half, out)
    whole_pre, pre = c.out(2 * half, dtype)
    L.moe_group_swiglu(c.x, c.offsets, c.w, h, pre=pre, src=c.src, src_div=c.div)
    gu = OG.matmul(c.xg, c.offsets_h, c.wf, c.rows)
    tol = _sum_tol(c.xg, c.wf, k, c.offsets_h, c.rows, OG.matmul)
    c.check(whole_pre, pre, gu, tol + _half_step(gu, dtype), "pre")
    (g, u), (tg, tu) = np.split(gu, 2, 1), np.split(tol, 2, 1)
    ref = OG.swiglu(gu)
    silu = g * OG.sigmoid(g)
    ht = 1.1 * tg * (np.abs(u) + tu) + np.abs(silu) * tu + np.abs(ref) * _silu_rel(g)
    c.check(whole, h, ref, ht + _half_step(ref, out), "h")
    whole2, h2 = c.out(half, out)
    L.moe_group_swiglu(c.x, c.offsets, c.w, h2, src=c.src, src_div=c.div)
    assert torch.equal(whole, whole2), "pre changes h"

    # down: w [n, k = half], dy [rows, n]
    n = k
    c = Case(counts, n, half, dtype, n, seed=half + 1, **VARIANTS[variant])
    rng = np.random.default_rng(half)
    pre = c.matrix(rng.standard_normal((c.rows, 2 * half)) * 2, dtype)
    whole, dpre = c.out(2 * half, out)
    L.moe_group_swiglu_grad(c.x, c.offsets, c.w, pre, dpre, src=c.src, src_div=c.div)
    dh = OG.matmul_t(c.xg, c.offsets_h, c.wf, c.rows)
    td = _sum_tol(c.xg, c.wf, n, c.offsets_h, c.rows, OG.matmul_t)
    ref = OG.swiglu_grad(dh, _f64(pre))
    one = np.abs(OG.swiglu_grad(np.ones_like(dh), _f64(pre)))
    g, u = np.split(_f64(pre), 2, 1)
    # s (1 + g (1 - s)): each factor's relative error on values below 1 + |g|
    factor = np.concatenate([np.abs(u) * (1 + np.abs(g)), np.abs(g)], 1) * np.tile(_silu_rel(g), 2)
    tol = np.tile(td, 2) * (one + factor) + np.tile(np.abs(dh), 2) * factor + _half_step(ref, out)
    c.check(whole, dpre, ref, tol, "dpre")


@pytest.mark.parametrize("variant", range(len(VARIANTS)))
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_weight_gradient(shape, dtype, out, variant):
    counts, n, k = SHAPES[shape]
    c = Case(counts, n, k, dtype, k, seed=shape, **VARIANTS[variant])
    rng = np.random.default_rng(shape)
    dy = c.matrix(rng.standard_normal((c.rows, n)), dtype)
    dw = torch.full((c.groups, n + 1, k + c.pad), SENTINEL, dtype=out, device="cuda")
    view = dw[:, :n, :k]
    L.moe_group_wgrad(dy, c.x, c.offsets, view, src=c.src, src_div=c.div)
    torch.cuda.synchronize()
    ref = OG.wgrad(_f64(dy), c.xg, c.offsets_h, c.groups)
    terms = np.array(counts)[:, None, None] + 2
    tol = terms * 2.0**-24 * OG.wgrad(np.abs(_f64(dy)), np.abs(c.xg), c.offsets_h, c.groups)
    _close(view, ref, tol + _half_step(ref, out), "dw")
    assert bool((dw[:, n:] == SENTINEL).all()) and bool((dw[:, :, k:] == SENTINEL).all())
    # accumulate: the fp32 sum plus what dw holds, one more half step of each
    held = _f64(view)
    L.moe_group_wgrad(dy, c.x, c.offsets, view, src=c.src, src_div=c.div, accumulate=True)
    torch.cuda.synchronize()
    _close(view, held + ref, tol + _half_step(held + ref, out) + np.abs(held + ref) * 2.0**-24, "dw +=")


def test_weight_gradient_without_rows_is_zero():
    dw = torch.full((3, 40, 24), SENTINEL, device="cuda")
    e = torch.empty((0, 40), dtype=BF16, device="cuda")
    x = torch.empty((0, 24), dtype=BF16, device="cuda")
    L.moe_group_wgrad(e, x, torch.zeros(4, dtype=torch.int32, device="cuda"), dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("n,k", [(64, 128), (33, 51)])
def test_operand_without_rows(n, k):
    """src given and no row that it could name: products and gradients of zeros."""
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    src = torch.tensor([-1, 0, 3, -1, 1], dtype=torch.int32, device="cuda")
    x, dy = (torch.empty((0, c), dtype=BF16, device="cuda") for c in (k, n))
    w = torch.ones((2, n, k), dtype=BF16, device="cuda")
    full = lambda *s: torch.full(s, SENTINEL, device="cuda")  # noqa: E731
    y, dx, dw, dpre = full(5, n), full(5, k), full(2, n, k), full(5, 2 * k)
    L.moe_group_matmul(x, off, w, y, src=src)
    L.moe_group_matmul_t(dy, off, w, dx, src=src)
    L.moe_group_swiglu_grad(dy, off, w, torch.ones((5, 2 * k), dtype=BF16, device="cuda"), dpre, src=src)
    L.moe_group_wgrad(torch.ones((5, n), dtype=BF16, device="cuda"), x, off, dw, src=src)
    for t in (y, dx, dpre, dw):
        assert bool((t == 0).all())


def test_values_that_are_not_finite_stay_in_their_rows():
    """A NaN or an infinity in one row of x, or past the columns of a strided operand, reaches that row alone."""
    c = Case([5, 9], 70, 100, BF16, 100, pad=4)
    base = c.x
    base[3, 50] = float("nan")
    base[9, 99] = float("inf")
    wide = torch.empty((c.rows, 104), dtype=BF16, device="cuda").fill_(float("nan"))
    wide[:, :100] = base
    whole, y = c.out(70, F32)
    L.moe_group_matmul(wide[:, :100], c.offsets, c.w, y)
    torch.cuda.synchronize()
    fine = torch.isfinite(y).all(1).cpu().numpy()
    assert not fine[3] and not fine[9] and fine[[i for i in range(14) if i not in (3, 9)]].all()
    # rows of no group may hold anything: they are not read into a group's gradient
    dy = torch.ones((c.rows, 70), dtype=BF16, device="cuda")
    x = torch.ones((c.rows, 100), dtype=BF16, device="cuda")
    dy[14:], x[14:] = float("nan"), float("inf")
    dw = torch.empty((2, 70, 100), device="cuda")
    L.moe_group_wgrad(dy, x, c.offsets, dw)
    assert bool((dw[0] == 5).all()) and bool((dw[1] == 9).all())


def test_offsets_out_of_range_are_clamped():
    c = Case([4, 4], 32, 64, BF16, 64, tail=0)
    for off in ([0, 4, 100], [-3, 4, 8], [6, 2, 8], [0, 2**31 - 1, 8], [8, 8, 8]):
        y = torch.full((8, 32), SENTINEL, device="cuda")
        L.moe_group_matmul(c.x, _dev(np.array(off, np.int32), torch.int32), c.w, y)
        ref = OG.matmul(c.xg, off, c.wf, 8)
        m = ~np.isnan(ref[:, 0])
        _close(y[torch.from_numpy(m).cuda()], ref[m], np.abs(ref[m]) * 1e-5 + 1e-5, str(off))
        assert bool((y[torch.from_numpy(~m).cuda()] == SENTINEL).all())


def test_offsets_that_do_not_ascend_write_inside():
    """Groups that overlap make more tiles than the grid holds: what is written stays inside y."""
    rows, groups = 200, 64
    off = torch.tensor([0, rows] * (groups // 2) + [0], dtype=torch.int32, device="cuda")
    x = torch.ones((rows, 64), dtype=BF16, device="cuda")
    w = torch.ones((groups, 40, 64), dtype=BF16, device="cuda")
    whole = torch.full((3 * rows, 40), SENTINEL, device="cuda")
    L.moe_group_matmul(x, off, w, whole[rows:2 * rows])
    assert bool((whole[:rows] == SENTINEL).all()) and bool((whole[2 * rows:] == SENTINEL).all())
    assert bool(((whole[rows:2 * rows] == 64) | (whole[rows:2 * rows] == SENTINEL)).all())


# ----------------------------------------------------------------------------- large
def _device_reference(way, x, w, bounds, src=None, div=1):
    """fp64 on the GPU: the same definitions for sizes that take the large tiles."""
    xs = x if src is None else x[(src.long() // div)]
    parts = []
    for g in range(len(bounds) - 1):
        a = xs[bounds[g]:bounds[g + 1]].double()
        parts.append(a @ (w[g].double() if way == "t" else w[g].double().t().contiguous()))
    return torch.cat(parts)


LARGE = [([2048, 0, 1700, 333], 4608, 520), ([600] * 8, 2304, 264), ([5000], 1536, 1032), ([40] * 96, 1280, 512)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", range(len(LARGE)))
def test_large_products_and_gradients(shape, gather):
    """Every call at sizes of many tiles, bf16, against fp64 products on the GPU: relative error of the whole
    within half a bf16 step (2^-8) and of fp32 outputs within T * 2^-24 for T terms of like size."""
    counts, n, k = LARGE[shape]
    gen = torch.Generator(device="cuda").manual_seed(shape)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    groups, rows = len(counts), sum(counts)
    bounds = np.concatenate([[0], np.cumsum(counts)]).tolist()
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    x, w, dy = r(rows // 2 if gather else rows, k), r(groups, n, k) * 0.05, r(rows, n)
    src = torch.randint(0, 2 * x.shape[0], (rows,), generator=gen, device="cuda").int() if gather else None
    kw = dict(src=src, src_div=2) if gather else {}

    def near(got, ref, tol):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= tol, err
        worst = float(((got.double() - ref).abs() / (ref.abs() + ref.abs().mean())).max())
        assert worst <= 4 * tol + 1e-5, worst

    y = torch.empty(rows, n, dtype=BF16, device="cuda")
    L.moe_group_matmul(x, off, w, y, **kw)
    ref = _device_reference("n", x, w, bounds, src, 2)
    near(y, ref, 2.0**-8)
    h, pre = torch.empty(rows, n // 2, dtype=BF16, device="cuda"), torch.empty_like(y)
    L.moe_group_swiglu(x, off, w, h, pre=pre, **kw)
    g, u = ref.chunk(2, 1)
    near(pre, ref, 2.0**-8)
    near(h, torch.nn.functional.silu(g) * u, 2.0**-8)
    dx = torch.empty(rows, k, device="cuda")
    L.moe_group_matmul_t(dy, off, w, dx)
    ref = _device_reference("t", dy, w, bounds)
    near(dx, ref, n * 2.0**-24)
    pre2, dpre = r(rows, 2 * k), torch.empty(rows, 2 * k, dtype=BF16, device="cuda")
    L.moe_group_swiglu_grad(dy, off, w, pre2, dpre)
    g, u = pre2.double().chunk(2, 1)
    s = torch.sigmoid(g)
    near(dpre, torch.cat([ref * u * (s + g * s * (1 - s)), ref * g * s], 1), 2.0**-8)
    dw = torch.empty(groups, n, k, device="cuda")
    L.moe_group_wgrad(dy, x, off, dw, **kw)
    xs = x if src is None else x[src.long() // 2]
    ref = torch.stack([dy[a:b].double().t().contiguous() @ xs[a:b].double() for a, b in zip(bounds, bounds[1:])])
    near(dw, ref, max(counts) * 2.0**-24)
    again = torch.empty_like(dw)
    L.moe_group_wgrad(dy, x, off, again, **kw)
    assert torch.equal(dw, again)


def test_operands_past_32_bit_offsets():
    """x and y of 4.9 GB, rows picked from both ends."""
    rows, wide, narrow = 600_000, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros(rows, wide, dtype=BF16, device="cuda")
    at = torch.tensor([0, 7, 262_143, 262_144, 524_287, 524_288, rows - 1], device="cuda")
    x[at] = torch.randn(len(at), wide, generator=gen, device="cuda").to(BF16)
    w = (torch.randn(2, narrow, wide, generator=gen, device="cuda") * 0.05).to(BF16)
    src, off = at.int(), torch.tensor([0, 3, len(at)], dtype=torch.int32, device="cuda")
    y = torch.empty(len(at), narrow, device="cuda")
    L.moe_group_matmul(x, off, w, y, src=src)
    ref = torch.cat([x[at[:3]].double() @ w[0].double().t().contiguous(), x[at[3:]].double() @ w[1].double().t().contiguous()])
    _close(y, _f64(ref), np.abs(_f64(ref)) * 1e-5 + wide * 2.0**-24 * 4, "gathered from far rows")
    # all rows: the whole x, then its gradients
    off = torch.tensor([0, 524_280, rows], dtype=torch.int32, device="cuda")
    y = torch.empty(rows, narrow, device="cuda")
    L.moe_group_matmul(x, off, w, y)
    group = (at >= 524_280).long()
    ref = torch.stack([w[g].double() @ x[i].double() for g, i in zip(group.tolist(), at.tolist())])
    _close(y[at], _f64(ref), np.abs(_f64(ref)) * 1e-5 + wide * 2.0**-24 * 4, "rows past 4 GB")
    assert int((y != 0).any(1).sum()) == len(at)
    dy = torch.zeros(rows, narrow, dtype=BF16, device="cuda")
    dy[at] = torch.randn(len(at), narrow, generator=gen, device="cuda").to(BF16)
    dw = torch.empty(2, narrow, wide, device="cuda")
    L.moe_group_wgrad(dy, x, off, dw)
    ref = torch.stack([dy[at][group == g].double().t().contiguous() @ x[at][group == g].double() for g in (0, 1)])
    _close(dw, _f64(ref), np.abs(_f64(ref)) * 1e-5 + 1e-5, "dw over 4 GB")
    out = torch.empty(rows, wide, dtype=BF16, device="cuda")
    L.moe_group_matmul_t(dy, off, w, out)
    ref = torch.stack([w[g].double().t().contiguous() @ dy[i].double() for g, i in zip(group.tolist(), at.tolist())])
    _close(out[at], _f64(ref), np.abs(_f64(ref)) * 2.0**-8 + 1e-4, "y past 4 GB")


def test_group_of_just_over_4_gib():
    """One group's rows, ungathered, of 2^32 bytes and ten rows more: its first tile holds whole rows all the same."""
    rows, wide, narrow = (1 << 19) + 10, 4096, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(rows, wide, dtype=BF16, device="cuda")
    at = torch.tensor([0, 9, 10, 100, 255, 256, 300, 524_287, rows - 1], device="cuda")
    x[at] = torch.randn(len(at), wide, generator=gen, device="cuda").to(BF16)
    w = (torch.randn(1, narrow, wide, generator=gen, device="cuda") * 0.05).to(BF16)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    for n in (narrow, 1):                        # 1: columns of another tile shape
        y = torch.empty(rows, n, device="cuda")
        L.moe_group_matmul(x, off, w[:, :n], y)
        ref = x[at].double() @ w[0, :n].double().t().contiguous()
        _close(y[at], _f64(ref), np.abs(_f64(ref)) * 1e-5 + wide * 2.0**-24 * 4, f"{n} columns")
        assert int((y != 0).any(1).sum()) == len(at)


def test_many_groups():
    """The largest number of groups, most of them empty."""
    groups, n, k = 1024, 72, 64
    counts = np.zeros(groups, np.int64)
    counts[[0, 1, 63, 64, 511, 700, 1023]] = [3, 70, 1, 130, 2, 5, 9]
    c = Case(counts.tolist(), n, k, BF16, k)
    whole, y = c.out(n, F32)
    L.moe_group_matmul(c.x, c.offsets, c.w, y)
    ref = OG.matmul(c.xg, c.offsets_h, c.wf, c.rows)
    c.check(whole, y, ref, _sum_tol(c.xg, c.wf, k, c.offsets_h, c.rows, OG.matmul) + _half_step(ref, F32), "1024 groups")


# ----------------------------------------------------------------------------- dispatch
@pytest.mark.parametrize("rows,top_k,groups", [(1, 1, 1), (8, 6, 384), (4, 2, 16), (341, 6, 384), (342, 6, 384), (1024, 2, 1),
                                               (1025, 2, 1024), (3000, 3, 7), (2731, 3, 128), (20000, 8, 1024), (0, 3, 5)])
def test_plan(rows, top_k, groups):
    rng = np.random.default_rng(rows + groups)
    idx = np.minimum((groups * rng.random((rows, top_k)) ** 3).astype(np.int32), groups - 1)
    flip = rng.random(idx.shape)
    idx[flip < 0.05], idx[flip > 0.98], idx[(flip > 0.97) & (flip < 0.98)] = -1, groups, -7
    offsets = torch.full((groups + 1,), 99, dtype=torch.int32, device="cuda")
    pairs, pos = (torch.full((rows * top_k,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    need = L.group_plan_bytes(rows, top_k, groups)
    ws = torch.randint(0, 255, (need,), dtype=torch.uint8, device="cuda") if need else None
    L.moe_group_plan(_dev(idx, torch.int32), groups, offsets, pairs, pos, ws)
    flat = idx.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    held = int((key < groups).sum())
    want = np.where(np.arange(len(flat)) < held, order, -1)
    place = np.where(flat == -1, -1, -2)
    place[order[:held]] = np.arange(held)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])]))
    assert np.array_equal(pairs.cpu().numpy(), want) and np.array_equal(pos.cpu().numpy(), place)
    if rows * top_k <= 64:
        for a, b in zip(OG.plan(idx, groups), (offsets, pairs, pos)):
            assert np.array_equal(a, b.cpu().numpy())


# ----------------------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16), (F32, BF16), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,top_k,n,pad", [(1, 1, 1, 0), (5, 6, 512, 0), (8, 3, 77, 0), (33, 8, 264, 8), (9, 2, 5120, 1),
                                              (700, 4, 1000, 0)])
def test_combine_and_its_gradients(rows, top_k, n, pad, dtype, out):
    rng = np.random.default_rng(rows + n)
    p = rows * top_k
    o_rows = p + 3

    def matrix(r, dt):
        whole = torch.full((r, n + pad), SENTINEL, dtype=dt, device="cuda")
        whole[:, :n] = _dev(rng.standard_normal((r, n)), dt)
        return whole, whole[:, :n]

    _, o = matrix(o_rows, dtype)
    pos = rng.permutation(o_rows)[:p].astype(np.int32)
    if p > 4:
        pos[2] = -1
    w = rng.random((rows, top_k)).astype(np.float32)
    wd, posd = _dev(w, F32), _dev(pos, torch.int32)
    for ps, wt in ((pos, w), (None, w), (pos, None)):
        whole, y = matrix(rows, out)
        L.moe_group_combine(o, None if ps is None else posd, None if wt is None else wd, y, top_k=top_k)
        ref = OG.combine(_f64(o), ps, wt, rows, top_k)
        size = OG.combine(np.abs(_f64(o)), ps, wt, rows, top_k)
        _close(y, ref, size * (top_k + 1) * 2.0**-24 + _half_step(ref, out), "combine")
        assert bool((whole[:, n:] == SENTINEL).all())
    _, dy = matrix(rows, dtype)
    _, d_o = matrix(o_rows, out)
    d_o.fill_(SENTINEL)
    d_w = torch.empty((rows, top_k), device="cuda")
    L.moe_group_combine_grad(dy, o, posd, wd, d_o, d_w)
    ref_o, ref_w = OG.combine_grad(_f64(dy), _f64(o), pos, w, top_k)
    named = ~np.isnan(ref_o[:, 0])
    rows_named = torch.from_numpy(named).cuda()
    _close(d_o[rows_named], ref_o[named], np.abs(ref_o[named]) * 2.0**-24 + _half_step(ref_o[named], out), "d_o")
    assert bool((d_o[~rows_named] == SENTINEL).all())
    size = OG.combine_grad(np.abs(_f64(dy)), np.abs(_f64(o)), pos, w, top_k)[1]
    _close(d_w, ref_w, size * (n + 1) * 2.0**-24 + 1e-30, "d_wts")
    only_w, only_o = torch.empty_like(d_w), d_o.clone().fill_(SENTINEL)
    L.moe_group_combine_grad(dy, o, posd, wd, None, only_w)
    L.moe_group_combine_grad(dy, None, posd, wd, only_o, None, top_k=top_k)
    assert torch.equal(only_w, d_w) and torch.equal(only_o, d_o)


def test_combine_places_outside():
    o = torch.ones((4, 24), dtype=BF16, device="cuda")
    pos = _dev(np.array([0, 4, -1, -1, -2, 1, 3, 2], np.int32), torch.int32)
    y = torch.empty((4, 24), device="cuda")
    L.moe_group_combine(o, pos, None, y, top_k=2)
    y = y.cpu().numpy()
    assert np.isnan(y[0]).all() and (y[1] == 0).all() and np.isnan(y[2]).all() and (y[3] == 2).all()
    d_w = torch.empty((4, 2), device="cuda")
    L.moe_group_combine_grad(torch.ones((4, 24), dtype=BF16, device="cuda"), o, pos, None, None, d_w)
    assert np.array_equal(d_w.cpu().numpy(), [[24, np.nan], [0, 0], [np.nan, 24], [24, 24]], equal_nan=True)


# ----------------------------------------------------------------------------- together
class Layer:
    """A routed SwiGLU layer of 16-bit experts, forward and backward, through the library's calls."""

    def __init__(self, rows=37, top_k=3, groups=6, hidden=136, inter=88, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.top_k, self.groups, self.rows = top_k, groups, rows
        r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
        self.x = r(rows, hidden).to(BF16).cuda()
        self.w1 = (r(groups, 2 * inter, hidden) * 0.1).to(BF16).cuda()
        self.w2 = (r(groups, hidden, inter) * 0.1).to(BF16).cuda()
        self.dy = r(rows, hidden).to(BF16).cuda()
        self.idx = torch.stack([torch.randperm(groups, generator=g)[:top_k] for _ in range(rows)]).int().cuda()
        self.wts = torch.softmax(r(rows, top_k), 1).float().cuda()
        p, dev = rows * top_k, "cuda"
        self.offsets = torch.empty(groups + 1, dtype=torch.int32, device=dev)
        self.pairs, self.pos = (torch.empty(p, dtype=torch.int32, device=dev) for _ in range(2))
        e = lambda *s, t=F32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
        self.h, self.pre, self.o = e(p, inter, t=BF16), e(p, 2 * inter, t=BF16), e(p, hidden, t=BF16)
        self.y, self.d_o, self.d_wts = e(rows, hidden), e(p, hidden, t=BF16), e(rows, top_k)
        self.dpre, self.dxp, self.dx = e(p, 2 * inter, t=BF16), e(p, hidden, t=BF16), e(rows, hidden)
        self.dw1, self.dw2 = e(groups, 2 * inter, hidden), e(groups, hidden, inter)

    def run(self):
        L.moe_group_plan(self.idx, self.groups, self.offsets, self.pairs, self.pos)
        L.moe_group_swiglu(self.x, self.offsets, self.w1, self.h, pre=self.pre, src=self.pairs, src_div=self.top_k)
        L.moe_group_matmul(self.h, self.offsets, self.w2, self.o)
        L.moe_group_combine(self.o, self.pos, self.wts, self.y)
        L.moe_group_combine_grad(self.dy, self.o, self.pos, self.wts, self.d_o, self.d_wts)
        L.moe_group_swiglu_grad(self.d_o, self.offsets, self.w2, self.pre, self.dpre)
        L.moe_group_wgrad(self.d_o, self.h, self.offsets, self.dw2)
        L.moe_group_wgrad(self.dpre, self.x, self.offsets, self.dw1, src=self.pairs, src_div=self.top_k)
        L.moe_group_matmul_t(self.dpre, self.offsets, self.w1, self.dxp)
        L.moe_group_combine(self.dxp, self.pos, None, self.dx)

    def results(self):
        return [self.y, self.d_wts, self.dw1, self.dw2, self.dx]

    def reference(self):
        """The same results by autograd in fp64 on the CPU (bf16 inputs, nothing rounded between)."""
        x, w1, w2, wts = (t.cpu().double().requires_grad_() for t in (self.x, self.w1, self.w2, self.wts))
        idx, y = self.idx.cpu().long(), 0
        for j in range(self.top_k):
            gu = torch.bmm(w1[idx[:, j]], x[:, :, None])[..., 0]
            g, u = gu.chunk(2, 1)
            y = y + wts[:, j:j + 1] * torch.bmm(w2[idx[:, j]], (torch.nn.functional.silu(g) * u)[:, :, None])[..., 0]
        (y * self.dy.cpu().double()).sum().backward()
        return [t.detach().numpy() for t in (y, wts.grad, w1.grad, w2.grad, x.grad)]


def _layer_matches(layer, ref):
    # bf16 at h, o, d_o, dpre, dxp: five roundings of 2^-9 rms each at most, summed as if aligned: 5 * 2^-8 of the norm
    for name, got, want in zip(("y", "d_wts", "dw1", "dw2", "dx"), layer.results(), ref):
        err = np.linalg.norm(_f64(got) - want) / np.linalg.norm(want)
        assert err <= 5 * 2.0**-8, f"{name}: {err:.3g}"


def test_layer_forward_and_backward():
    layer = Layer()
    layer.run()
    torch.cuda.synchronize()
    _layer_matches(layer, layer.reference())
    first = [t.clone() for t in layer.results()]
    layer.run()
    assert all(torch.equal(a, b) for a, b in zip(first, layer.results())), "not the same bits twice"


def test_layer_captured_and_replayed():
    layer, other = Layer(seed=1), Layer(seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for turn in range(4):
        src = Layer(seed=10 + turn)
        for a in ("x", "w1", "w2", "dy", "idx", "wts"):
            getattr(layer, a).copy_(getattr(src, a))
        for t in layer.results():
            t.fill_(SENTINEL)
        graph.replay()
        other.run()                                      # eager work between the replays
        torch.cuda.synchronize()
        src.run()
        assert all(torch.equal(a, b) for a, b in zip(layer.results(), src.results())), turn
        _layer_matches(layer, src.reference())


def test_two_streams_at_once():
    layers = [Layer(rows=300, seed=s) for s in (3, 4)]
    for l in layers:
        l.run()
    want = [[t.clone() for t in l.results()] for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        for l, s in zip(layers, streams):
            with torch.cuda.stream(s):
                l.run()
    torch.cuda.synchronize()
    for l, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(l.results(), w))


def test_binding_refuses():
    c = Case([4, 4], 32, 64, BF16, 64, tail=0)
    y = torch.empty((8, 32), device="cuda")
    cases = [lambda: L.moe_group_matmul(c.x[:, :63], c.offsets, c.w, y),
             lambda: L.moe_group_matmul(c.x.float(), c.offsets, c.w.float(), y),
             lambda: L.moe_group_matmul(c.x.half(), c.offsets, c.w, y),
             lambda: L.moe_group_matmul(c.x, c.offsets.long(), c.w, y),
             lambda: L.moe_group_matmul(c.x, c.offsets[:2], c.w, y),
             lambda: L.moe_group_matmul(c.x[:7], c.offsets, c.w, y),
             lambda: L.moe_group_matmul(c.x, c.offsets, c.w.transpose(1, 2), y),
             lambda: L.moe_group_matmul(c.x, c.offsets, c.w, y.t()),
             lambda: L.moe_group_matmul(c.x, c.offsets, c.w, y.double()),
             lambda: L.moe_group_matmul(c.x, c.offsets, c.w, y, src=c.offsets),
             lambda: L.moe_group_swiglu(c.x, c.offsets, c.w, y),
             lambda: L.moe_group_swiglu_grad(c.x, c.offsets, c.w, None, y),
             lambda: L.moe_group_wgrad(c.x, c.x[:4], c.offsets, c.w),
             lambda: L.moe_group_wgrad(c.x, c.x, c.offsets, torch.empty((1, 64, 64), device="cuda").expand(2, 64, 64)),
             lambda: L.moe_group_combine(c.x, None, None, y),
             lambda: L.moe_group_plan(c.offsets[None], 4, c.offsets, c.offsets, c.offsets)]
    for i, f in enumerate(cases):
        with pytest.raises(L.MoeError):
            f()
            pytest.fail(f"case {i} was taken")
