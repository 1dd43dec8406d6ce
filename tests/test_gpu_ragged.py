"""Grouped matrix products, their gradients, the INT8 products and SwiGLU against plain 64-bit formulas.

Tolerances, per element, from the number formats:
  - a product's accumulation: each tensor-core instruction adds 16 products to the running FP32 sum and
    truncates, which loses less than two units of its last place, 2^-22 of S = sum |a||b|; fp32 results
    are flushed or cut at least every 256 instructions; segments, split and join sums are FP32 additions,
    each within 2^-24 of S;
  - the result's rounding: half a step, torch.finfo(t).eps / 2 of its magnitude (and half the smallest
    subnormal of fp16).
INT8 sums are exact; their scaling is three FP32 roundings.
"""
import numpy as np
import pytest
import torch

import group_limited_routing_router_b200 as bm

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
D = torch.float64


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int64, device="cuda")


def spans(counts, first=0):
    at = first
    for e, c in enumerate(counts):
        if c:
            yield e, at, at + c
        at += c


def half_step(want, dtype):
    tiny = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -150}[dtype]
    return want.abs() * (torch.finfo(dtype).eps / 2) + tiny


def sum_tol(mag, length, dtype):
    """Bound of the accumulation error of `length` products of summed magnitude `mag`."""
    instructions = length // 16 + 1
    if dtype == F32:
        instructions = min(instructions, 256)
    segments = length // 256 + 1  # the shortest cut, of fp32 results: 256 products
    return mag * (instructions * 2.0 ** -22 + (segments + 72) * 2.0 ** -24)


def check(got, want, tol, what):
    bad = ~((got.to(D) - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{((got.to(D) - want).abs() / tol.clamp_min(1e-300)).max().item():.3g} of the tolerance"


def status_ok():
    torch.cuda.synchronize()
    assert bm.device_status() == bm.OK


def ragged_counts(E, R, seed, empty=0.2):
    r = np.random.RandomState(seed)
    p = np.exp(r.standard_normal(E)) * (r.rand(E) >= empty)
    if p.sum() == 0:
        p[0] = 1
    return r.multinomial(R, p / p.sum())


def products(x, dy, w, counts, first=0):
    """The three products and their magnitudes in 64 bits: {name: (value, sum of magnitudes)}."""
    E, N, K = w.shape
    R = x.shape[0]
    z = lambda *s: torch.zeros(*s, dtype=D, device="cuda")  # noqa: E731
    out = dict(out=(z(R, N), z(R, N)), dx=(z(R, K), z(R, K)), dw=(z(E, N, K), z(E, N, K)))
    for e, a, b in spans(counts, first):
        xe, de, we = x[a:b].to(D), dy[a:b].to(D), w[e].to(D)
        for i, f in enumerate((lambda t: t, torch.abs)):
            out["out"][i][a:b] = f(xe) @ f(we).t()
            out["dx"][i][a:b] = f(de) @ f(we)
            out["dw"][i][e] = f(de).t() @ f(xe)
    return out


def run_all(x, dy, w, off, dtype):
    return dict(out=bm.grouped_mm(x, w, off, out_dtype=dtype), dx=bm.grouped_mm_dgrad(dy, w, off, out_dtype=dtype),
                dw=bm.grouped_mm_wgrad(dy, x, off, out_dtype=dtype))


def check_all(got, ref, N, K, counts, dtype, what):
    rows = max(1, int(max(counts)) if len(counts) else 1)
    for name, length in (("out", K), ("dx", N), ("dw", rows)):
        v, mag = ref[name]
        check(got[name], v, half_step(v, dtype) + sum_tol(mag, length, dtype), f"{what} {name}")


CASES = [  # E, rows, K, N: each kernel, each tile edge
    (1, 1, 64, 64), (1, 1, 8, 8), (1, 7, 72, 136), (2, 5, 64, 128), (3, 40, 320, 192), (4, 333, 512, 384),
    (16, 16, 1024, 512), (16, 1501, 320, 192), (5, 2000, 264, 520), (8, 4096, 640, 1280), (64, 700, 256, 128),
    (256, 300, 128, 256), (256, 2048, 64, 72), (1, 257, 2560, 264), (1, 6000, 128, 248), (2, 3000, 1000, 2056),
    (37, 12000, 520, 1032), (2, 9000, 2040, 520), (2, 9000, 520, 2040),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("E,R,K,N", CASES)
def test_products_and_gradients(E, R, K, N, dtype):
    g = gen(E * 1000 + R)
    counts = ragged_counts(E, R, R + E)
    x, dy, w = normal(g, R, K, dtype=dtype), normal(g, R, N, dtype=dtype), normal(g, E, N, K, dtype=dtype,
                                                                                scale=K ** -0.5)
    off = offsets_of(counts)
    ref = products(x, dy, w, counts)
    for out_dtype in (dtype, F32):
        got = run_all(x, dy, w, off, out_dtype)
        status_ok()
        check_all(got, ref, N, K, counts, out_dtype, f"{out_dtype}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("E,R,K,N", [(1, 12000, 1032, 2056), (1, 12000, 2056, 1032), (32, 20000, 776, 1544),
                                     (8, 20000, 1032, 2056), (4, 3000, 2568, 264), (1, 2100, 520, 2312)])
def test_bands_of_row_tiles(E, R, K, N, dtype):
    """Groups of many row tiles (whole and cut bands of them) over several feature tiles, two per pair among them;
    few items on the pairs."""
    g = gen(R + N)
    counts = ragged_counts(E, R, N)
    x, dy, w = normal(g, R, K, dtype=dtype), normal(g, R, N, dtype=dtype), normal(g, E, N, K, dtype=dtype,
                                                                                scale=K ** -0.5)
    off = offsets_of(counts)
    ref = products(x, dy, w, counts)
    got = dict(out=bm.grouped_mm(x, w, off), dx=bm.grouped_mm_dgrad(dy, w, off))
    status_ok()
    for name, length in (("out", K), ("dx", N)):
        v, mag = ref[name]
        check(got[name], v, half_step(v, dtype) + sum_tol(mag, length, dtype), name)


@pytest.mark.parametrize("mean", [1, 12, 33, 64, 130, 400])
def test_every_group_size(mean):
    """Groups of every size around the tiles' edges, empty ones among them."""
    E, K, N = 96, 192, 320
    r = np.random.RandomState(mean)
    counts = r.randint(0, 2 * mean + 1, size=E)
    counts[:4] = [0, 1, mean, 2 * mean]
    R = int(counts.sum())
    g = gen(mean)
    x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, E, N, K, scale=K ** -0.5)
    got = run_all(x, dy, w, offsets_of(counts), BF)
    status_ok()
    check_all(got, products(x, dy, w, counts), N, K, counts, BF, f"mean {mean}")


@pytest.mark.parametrize("E,R", [(4, 40), (4, 600), (2, 3000)])
def test_rows_outside_the_groups(E, R):
    """Rows before the first and behind the last group hold NaN: nothing reads them into a sum, nothing
    writes their outputs; the rows of one group do not reach the next one's sums."""
    K, N, first, behind = 136, 200, 9, 37
    g = gen(R)
    counts = ragged_counts(E, R, 3, empty=0.0)
    total = first + R + behind
    x, dy, w = normal(g, total, K), normal(g, total, N), normal(g, E, N, K, scale=K ** -0.5)
    ref = products(x, dy, w, counts, first)
    for t in (x, dy):
        t[:first] = float("nan")
        t[first + R:] = float("nan")
    off = offsets_of(counts, first)
    out = torch.full((total, N), 7.0, dtype=BF, device="cuda")
    dx = torch.full((total, K), 7.0, dtype=BF, device="cuda")
    bm.grouped_mm(x, w, off, out=out)
    bm.grouped_mm_dgrad(dy, w, off, out=dx)
    dw = bm.grouped_mm_wgrad(dy, x, off)
    status_ok()
    for t in (out, dx):
        assert (t[:first] == 7).all() and (t[first + R:] == 7).all()
    inside = slice(first, first + R)
    ref = {k: (v if k == "dw" else (v[0][inside], v[1][inside])) for k, v in ref.items()}
    check_all(dict(out=out[inside], dx=dx[inside], dw=dw), ref, N, K, counts, BF, "inside")


def test_a_groups_infinities_stay_its_own():
    E, K, N = 3, 128, 192
    counts = [37, 21, 50]
    g = gen(5)
    x, dy, w = normal(g, 108, K), normal(g, 108, N), normal(g, E, N, K)
    clean = run_all(x, dy, w, offsets_of(counts), BF)
    x2, dy2 = x.clone(), dy.clone()
    x2[37:58] = float("inf")
    dy2[37:58] = float("nan")
    got = run_all(x2, dy2, w, offsets_of(counts), BF)
    status_ok()
    for k in ("out", "dx"):
        assert torch.equal(got[k][:37], clean[k][:37]) and torch.equal(got[k][58:], clean[k][58:])
    assert torch.equal(got["dw"][0], clean["dw"][0]) and torch.equal(got["dw"][2], clean["dw"][2])
    assert got["dw"][1].isnan().all()


@pytest.mark.parametrize("R,E", [(24, 3), (700, 3), (9000, 2)])
def test_strided_rows(R, E):
    """x, dy and the outputs as column blocks of wider buffers; the columns beside them stay."""
    K, N = 128, 256
    g = gen(R)
    counts = ragged_counts(E, R, 1)
    xb, db = normal(g, R, K + 72), normal(g, R, N + 8)
    x, dy, w = xb[:, 64:64 + K], db[:, :N], normal(g, E, N, K, scale=K ** -0.5)
    ob = torch.full((R, N + 24), 3.0, dtype=BF, device="cuda")
    gb = torch.full((R, K + 16), 3.0, dtype=F32, device="cuda")
    off = offsets_of(counts)
    out = bm.grouped_mm(x, w, off, out=ob[:, 16:16 + N])
    dx = bm.grouped_mm_dgrad(dy, w, off, out=gb[:, 8:8 + K], out_dtype=F32)
    dw = bm.grouped_mm_wgrad(dy, x, off)
    status_ok()
    ref = products(x, dy, w, counts)
    check(out, ref["out"][0], half_step(ref["out"][0], BF) + sum_tol(ref["out"][1], K, BF), "out")
    check(dx, ref["dx"][0], half_step(ref["dx"][0], F32) + sum_tol(ref["dx"][1], N, F32), "dx")
    check(dw, ref["dw"][0], half_step(ref["dw"][0], BF) + sum_tol(ref["dw"][1], R, BF), "dw")
    assert (ob[:, :16] == 3).all() and (ob[:, 16 + N:] == 3).all()
    assert (gb[:, :8] == 3).all() and (gb[:, 8 + K:] == 3).all()


@pytest.mark.parametrize("E,R,N,K", [(6, 300, 128, 192), (1, 20000, 192, 320), (2, 9000, 64, 72)])
def test_weight_gradient_accumulates(E, R, N, K):
    """accumulate adds to what is there, with and without split rows; an empty expert keeps its gradient."""
    g = gen(N)
    counts = ragged_counts(E, R, 2, empty=0.0)
    if E > 2:
        counts[1] += counts[3]
        counts[3] = 0
    dy, x = normal(g, R, N), normal(g, R, K)
    before = torch.randn(E, N, K, generator=g, device="cuda")
    dw = before.clone()
    assert bm.grouped_mm_wgrad(dy, x, offsets_of(counts), out=dw, accumulate=True) is dw
    status_ok()
    v, mag = products(x, dy, torch.zeros(E, N, K, device="cuda"), counts)["dw"]
    want = before.to(D) + v
    check(dw, want, half_step(want, F32) + sum_tol(mag, R, F32), "dw")
    if E > 2:
        assert torch.equal(dw[3], before[3])


@pytest.mark.parametrize("counts,N,K", [([0, 20000, 0], 192, 320), ([9000, 0], 64, 72), ([3, 0, 4], 192, 320),
                                        ([0, 9000], 4600, 1016)])
def test_an_expert_without_rows_keeps_every_bit(counts, N, K):
    """Negative zeros, NaN and subnormals of its accumulated gradient, with rows split and not."""
    g = gen(N)
    off = offsets_of(counts)
    dw = torch.randn(len(counts), N, K, generator=g, device="cuda")
    dw[:, ::2, ::3], dw[:, 1::2, 1::3], dw[:, :, 2::3] = -0.0, float("nan"), -1e-42
    before = dw.clone()
    bm.grouped_mm_wgrad(normal(g, sum(counts), N), normal(g, sum(counts), K), off, out=dw, accumulate=True)
    status_ok()
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e].view(torch.int32), before[e].view(torch.int32))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts", [[0, 5107, 300], [5107], [64, 0, 0, 6001]])
def test_weight_gradient_of_long_groups(counts, dtype):
    """The 512-column tiles: groups of more rows than one flush of fp32 results (4096) beside empty ones."""
    E, R, N, K = len(counts), sum(counts), 1016, 2568
    g = gen(R)
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    off = offsets_of(counts)
    v, mag = products(x, dy, torch.zeros(E, N, K, device="cuda"), counts)["dw"]
    for out_dtype in (dtype, F32):
        check(bm.grouped_mm_wgrad(dy, x, off, out_dtype=out_dtype), v,
              half_step(v, out_dtype) + sum_tol(mag, max(counts), out_dtype), f"{out_dtype}")
    before = torch.randn(E, N, K, generator=g, device="cuda")
    dw = before.clone()
    bm.grouped_mm_wgrad(dy, x, off, out=dw, accumulate=True)
    want = before.to(D) + v
    check(dw, want, half_step(want, F32) + sum_tol(mag + before.abs(), max(counts), F32), "accumulated")
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e], before[e])
    status_ok()


@pytest.mark.parametrize("N,K", [(256, 1280), (520, 264)])
def test_cleared_rows_of_many_short_groups(N, K):
    """Every length of a last k-step, on both CTAs of a pair, with NaN in every other group: a sum that met a row
    before it was cleared would be NaN."""
    counts = [1 + (i * 37) % 190 for i in range(256)]
    R = sum(counts)
    g = gen(K)
    dy, x = normal(g, R, N), normal(g, R, K)
    v, mag = products(x, dy, torch.zeros(256, N, K, device="cuda"), counts)["dw"]
    for e, a, b in spans(counts):
        if e % 2:
            dy[a:b] = float("nan")
            x[a:b] = float("nan")
    off = offsets_of(counts)
    first = None
    for _ in range(10):
        dw = bm.grouped_mm_wgrad(dy, x, off)
        check(dw[::2], v[::2], half_step(v[::2], BF) + sum_tol(mag[::2], max(counts), BF), "dw")
        first = dw if first is None else first
        assert torch.equal(dw[::2], first[::2]) and dw[1::2].isnan().all()
    status_ok()


def one_signed(g, *shape, dtype=BF):
    """Values in [1/2, 1]: sums of their products grow evenly, where truncation takes off the most."""
    return (torch.rand(*shape, generator=g, device="cuda") / 2 + 0.5).to(dtype)


def even_tol(want, piece, length):
    """Error of an evenly growing sum of `length` products in pieces of `piece`: an instruction truncates less than
    2^-22 of its running sum, half the piece's on average (a quarter more for its uneven growth); the pieces, and
    up to 64 partial sums of split contractions, are added in FP32."""
    m = min(piece, length) // 16 + 1
    return want * ((m / 2 + 1) * 1.25 * 2.0 ** -22 + (length // piece + 66) * 2.0 ** -24)


@pytest.mark.parametrize("E,R,K,N", [
    (1, 3000, 20480, 1024),  # CTA pairs
    (4, 40, 20480, 264),     # clusters that split the contraction, 32-row tiles
    (1, 300, 20480, 512),    # the same with 128-row tiles
    (64, 2048, 5120, 5120),  # one CTA per tile
])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_fp32_results_are_summed_in_short_pieces(E, R, K, N, dtype):
    """In one piece, 20480 one-signed products would come out 1280 x 2^-25 = 3.8e-5 low, 5120 of them 9.5e-6; the
    bounds are 1.2e-5 and 8.0e-6."""
    g = gen(R)
    counts = ragged_counts(E, R, 5)
    off = offsets_of(counts)
    x, w = one_signed(g, R, K, dtype=dtype), one_signed(g, E, N, K, dtype=dtype)
    out = bm.grouped_mm(x, w, off, out_dtype=F32)
    dx = bm.grouped_mm_dgrad(x, w.transpose(1, 2).contiguous(), off, out_dtype=F32)
    status_ok()
    want = torch.empty(R, N, dtype=D, device="cuda")
    for e, a, b in spans(counts):
        want[a:b] = x[a:b].to(D) @ w[e].to(D).t()
    check(out, want, even_tol(want, 256, K), "out")
    check(dx, want, even_tol(want, 256, K), "dx")


@pytest.mark.parametrize("counts,N,K,piece", [
    ([40000], 9456, 1016, 4096),      # 512-column tiles: 148 tiles of 256 columns on 74 pairs, 74 of 512
    ([64, 40000], 4600, 1016, 4096),  # 144 and 72
    ([40000, 3], 320, 192, 256),      # rows split over the pairs
    ([12000] * 8, 2560, 256, 256),    # 256-column tiles: K has no second 256
])
def test_fp32_weight_gradients_are_summed_in_pieces(counts, N, K, piece):
    """40000 one-signed rows in one piece would come out 2500 x 2^-25 = 7.5e-5 low, 12000 of them 2.2e-5; the bounds are
    4.3e-5 in pieces of 4096 and 9.5e-6 (12000 rows) in pieces of 256.  Accumulated ones take one rounding more per
    piece."""
    g = gen(N)
    R = sum(counts)
    off = offsets_of(counts)
    dy, x = one_signed(g, R, N), one_signed(g, R, K)
    want = torch.empty(len(counts), N, K, dtype=D, device="cuda")
    for e, a, b in spans(counts):
        want[e] = dy[a:b].to(D).t() @ x[a:b].to(D)
    dw = bm.grouped_mm_wgrad(dy, x, off, out_dtype=F32)
    status_ok()
    length = torch.tensor(counts, device="cuda")[:, None, None]
    tol = torch.stack([even_tol(want[e], piece, c) for e, c in enumerate(counts)])
    check(dw, want, tol, "dw")
    before = torch.rand(len(counts), N, K, generator=g, device="cuda") * length
    got = before.clone()
    bm.grouped_mm_wgrad(dy, x, off, out=got, accumulate=True)
    status_ok()
    want = want + before.to(D)
    check(got, want, tol + want * ((max(counts) // piece + 2) * 2.0 ** -24), "accumulated")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,N,K", [([5107], 9456, 1016), ([64, 5000], 4600, 1016), ([64, 0, 0, 6001], 2296, 1016),
                                        ([16384], 9456, 1016), ([0, 4097, 1, 63], 2296, 1016)])
def test_weight_gradient_on_512_column_tiles(counts, N, K, dtype):
    """Sizes whose 256-column tiles take two rounds of the 74 pairs and whose 512-column tiles take one, so that the
    latter run (one round costs 1060 cycles per k-step, two 1380; of the last, with 17 k-steps per group, only the
    16-bit result): one group, short and empty groups beside long ones, the longest single piece of fp16."""
    E, R = len(counts), sum(counts)
    g = gen(R)
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    off = offsets_of(counts)
    v, mag = products(x, dy, torch.zeros(E, N, K, device="cuda"), counts)["dw"]
    for out_dtype in (dtype, F32):
        check(bm.grouped_mm_wgrad(dy, x, off, out_dtype=out_dtype), v,
              half_step(v, out_dtype) + sum_tol(mag, max(counts), out_dtype), f"{out_dtype}")
    before = torch.randn(E, N, K, generator=g, device="cuda")
    dw = before.clone()
    bm.grouped_mm_wgrad(dy, x, off, out=dw, accumulate=True)
    want = before.to(D) + v
    check(dw, want, half_step(want, F32) + sum_tol(mag + before.abs(), max(counts), F32), "accumulated")
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(dw[e], before[e])
    status_ok()


def test_gradients_against_differences():
    """out is linear in x and in w: the change of sum(dy * out) along any direction is its gradient times
    that direction, exactly but for the roundings (fp32 results)."""
    E, R, K, N = 3, 90, 64, 96
    g = gen(11)
    counts = [40, 0, 50]
    x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, E, N, K)
    vx, vw = normal(g, R, K), normal(g, E, N, K)
    off = offsets_of(counts)
    f = lambda a, b: (bm.grouped_mm(a, b, off, out_dtype=F32).to(D) * dy.to(D)).sum()  # noqa: E731
    dx = bm.grouped_mm_dgrad(dy, w, off, out_dtype=F32).to(D)
    dw = bm.grouped_mm_wgrad(dy, x, off, out_dtype=F32).to(D)
    for got, grad, v in ((f(vx, w), dx, vx.to(D)), (f(x, vw), dw, vw.to(D))):
        want = (grad * v).sum()
        # both sides: 90 x 96 (or 3 x 64 x 96) terms of relative error below 2^-15 of their magnitudes
        assert abs(got - want) <= 2.0 ** -15 * (grad.abs() * v.abs()).sum() + 2.0 ** -15 * R * N * 8.0
    status_ok()


def test_bits_do_not_depend_on_the_run():
    g = gen(8)
    for E, R, K, N in ((16, 40, 2048, 256), (4, 900, 512, 512), (1, 30000, 128, 128)):
        counts = ragged_counts(E, R, 4)
        x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, E, N, K)
        off = offsets_of(counts)
        one = run_all(x, dy, w, off, F32)
        for _ in range(3):
            two = run_all(x, dy, w, off, F32)
            assert all(torch.equal(one[k], two[k]) for k in one)
    status_ok()


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [-1, 4, 8, 20], [0, 4, 8, 21]])
def test_bad_offsets_write_nothing(bad):
    R, K, N = 20, 64, 64
    g = gen(1)
    x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, 3, N, K)
    off = torch.tensor(bad, dtype=torch.int64, device="cuda")
    for call, shape in ((lambda o: bm.grouped_mm(x, w, off, out=o), (R, N)),
                        (lambda o: bm.grouped_mm_dgrad(dy, w, off, out=o), (R, K)),
                        (lambda o: bm.grouped_mm_wgrad(dy, x, off, out=o), (3, N, K))):
        out = torch.full(shape, 5.0, dtype=BF, device="cuda")
        call(out)
        torch.cuda.synchronize()
        assert bm.device_status() == bm.ERR_BAD_INDEX
        assert (out == 5).all()
    status_ok()


def test_bad_offsets_with_split_rows_write_nothing():
    R = 9000
    g = gen(2)
    x, dy = normal(g, R, 64), normal(g, R, 64)
    out = torch.full((2, 64, 64), 5.0, dtype=BF, device="cuda")
    bm.grouped_mm_wgrad(dy, x, torch.tensor([0, R + 1, R], device="cuda"), out=out)
    torch.cuda.synchronize()
    assert bm.device_status() == bm.ERR_BAD_INDEX and (out == 5).all()


def test_no_rows():
    w = normal(gen(1), 3, 64, 128)
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    x, dy = torch.empty(0, 128, dtype=BF, device="cuda"), torch.empty(0, 64, dtype=BF, device="cuda")
    assert bm.grouped_mm(x, w, off).shape == (0, 64)
    assert bm.grouped_mm_dgrad(dy, w, off).shape == (0, 128)
    assert (bm.grouped_mm_wgrad(dy, x, off) == 0).all()
    keep = torch.ones(3, 64, 128, device="cuda")
    bm.grouped_mm_wgrad(dy, x, off, out=keep, accumulate=True)
    assert (keep == 1).all()
    q, s = bm.quant_i8_rows(x)
    assert q.shape == (0, 128) and s.shape == (0,)
    assert bm.swiglu(x, x).shape == (0, 128)
    # rows, but no group has one
    x, dy = normal(gen(2), 30, 128), normal(gen(3), 30, 64)
    out = torch.full((30, 64), 2.0, dtype=BF, device="cuda")
    bm.grouped_mm(x, w, off, out=out)
    assert (out == 2).all() and (bm.grouped_mm_wgrad(dy, x, off) == 0).all()
    status_ok()


# ---- INT8 -------------------------------------------------------------------------------------------
def i8_operands(g, E, R, K, N):
    q = torch.randint(-128, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    return q, torch.rand(R, generator=g, device="cuda") + 0.1, w, (torch.rand(E, N, generator=g, device="cuda") + 0.1)


I8_CASES = [(1, 1, 16, 16), (1, 1, 5120, 640), (1, 17, 144, 272), (3, 40, 320, 192), (64, 80, 512, 256),
            (16, 1501, 320, 192), (1, 300, 2560, 528), (1, 5000, 640, 2560), (8, 9000, 528, 2064),
            (2, 9000, 1168, 2032)]


@pytest.mark.parametrize("out_dtype", [BF, HF, F32])
@pytest.mark.parametrize("E,R,K,N", I8_CASES)
def test_int8_product(E, R, K, N, out_dtype):
    """Every code, -128 among them; the sums are exact and the scaling three FP32 roundings."""
    g = gen(R + K)
    q, rs, w, cs = i8_operands(g, E, R, K, N)
    if out_dtype == HF:
        rs = rs * (1.0 / K)
    counts = ragged_counts(E, R, K)
    out = bm.grouped_mm_i8(q, rs, w, cs, offsets_of(counts), out_dtype=out_dtype)
    status_ok()
    want = torch.zeros(R, N, dtype=D, device="cuda")
    for e, a, b in spans(counts):
        want[a:b] = (q[a:b].to(D) @ w[e].to(D).t()) * rs[a:b].to(D)[:, None] * cs[e].to(D)
    check(out, want, half_step(want, out_dtype) + want.abs() * (3 * 2.0 ** -24 * 1.01), f"{out_dtype}")


@pytest.mark.parametrize("out_dtype", [BF, HF, F32])
@pytest.mark.parametrize("E,R,K,N", [(4, 3000, 2560, 272), (1, 12000, 144, 1040), (1, 2100, 528, 2320)])
def test_int8_results_keep_to_their_columns(E, R, K, N, out_dtype):
    """Results in a wider tensor's columns, rows in bands: what lies beside them stays."""
    g = gen(R + K)
    q, rs, w, cs = i8_operands(g, E, R, K, N)
    rs = rs * (1.0 / K)
    counts = ragged_counts(E, R, K)
    wide = torch.full((R, N + 48), 3.0, dtype=out_dtype, device="cuda")
    bm.grouped_mm_i8(q, rs, w, cs, offsets_of(counts), out=wide[:, 16:16 + N])
    status_ok()
    assert (wide[:, :16] == 3).all() and (wide[:, 16 + N:] == 3).all()
    want = torch.zeros(R, N, dtype=D, device="cuda")
    for e, a, b in spans(counts):
        want[a:b] = (q[a:b].to(D) @ w[e].to(D).t()) * rs[a:b].to(D)[:, None] * cs[e].to(D)
    check(wide[:, 16:16 + N], want, half_step(want, out_dtype) + want.abs() * (3 * 2.0 ** -24 * 1.01), f"{out_dtype}")


def test_int8_largest_sums():
    """65536 products of -128 and -128: 2^30, exact in INT32."""
    K = 65536
    q = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((16, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(2, device="cuda"), torch.ones(16, device="cuda")
    out = bm.grouped_mm_i8(q, one[0], w, one[1], out_dtype=F32)
    assert (out == 2.0 ** 30).all()
    status_ok()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,K", [(1, 8), (3, 64), (77, 1024), (5, 1032), (33, 5120), (2, 16384), (2, 65536)])
def test_row_quantiser(R, K, dtype):
    g = gen(K)
    x = normal(g, R, K, dtype=dtype, scale=3.0)
    x[0] = 0
    if R > 1:
        x[1, K // 2] = float("inf")
    if R > 2:
        x[2, K // 3] = float("nan")
    q, s = bm.quant_i8_rows(x)
    status_ok()
    f = x.float()
    # by a tensor: torch multiplies by the reciprocal of a Python number, which is another rounding
    want = f.abs().amax(dim=1) / torch.full((R,), 127.0, device="cuda")
    assert torch.equal(s.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    codes = torch.round(f / want[:, None])
    codes[~(want.isfinite() & (want > 0))] = 0
    assert torch.equal(q, codes.to(torch.int8))


@pytest.mark.parametrize("scale", [1e-44, 1e-37, 2.0 ** -98, 1.0, 1e30, 2e38])
def test_row_quantiser_rounds_every_quotient(scale):
    """Rows made of the neighbourhoods of the ties: multiples of half a code and the floats beside them, for
    scales from the subnormals to the largest; the codes are those of CUDA's own division."""
    g = gen(77)
    most = torch.rand(200, 1, generator=g, device="cuda") + 1.0
    halves = torch.arange(-254, 255, device="cuda") / 2.0
    x = (most / 127.0) * halves[None, :]
    x = torch.cat([x, torch.nextafter(x, x + 1), torch.nextafter(x, x - 1), most, x[:, :8] * 0], dim=1) * scale
    x = x.float()
    q, s = bm.quant_i8_rows(x)
    status_ok()
    want = x.abs().amax(dim=1) / torch.full((200,), 127.0, device="cuda")
    assert torch.equal(s, want)
    codes = torch.round(x / want[:, None]).clamp(-127, 127)
    codes[want == 0] = 0
    assert torch.equal(q, codes.to(torch.int8))


def test_quantised_rows_with_infinities_give_nan():
    g = gen(4)
    x = normal(g, 4, 64)
    x[1, 3], x[2, 5] = float("-inf"), float("nan")
    q, s = bm.quant_i8_rows(x)
    w = torch.randint(-127, 128, (32, 64), generator=g, device="cuda", dtype=torch.int8)
    out = bm.grouped_mm_i8(q, s, w, torch.ones(32, device="cuda"))
    assert out[1:3].isnan().all() and out[0].isfinite().all() and out[3].isfinite().all()
    status_ok()


# ---- SwiGLU -----------------------------------------------------------------------------------------
def swiglu_ref(dh, g, u):
    dh, g, u = dh.to(D), g.to(D), u.to(D)
    s = torch.sigmoid(g)
    return g * s * u, dh * u * s * (1 + g * (1 - s)), dh * g * s


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,I", [(1, 8), (77, 192), (300, 2560), (5, 5128), (70000, 16)])
def test_swiglu_and_gradient(R, I, dtype):
    """FP32 arithmetic: sigma within 6 roundings (exp within 2 of its argument's product, the sum, the
    quotient), the rest below 6 more; 1 + g (1 - sigma) cancels near g = -1.28, so dg's bound takes its
    terms' magnitudes."""
    rng = gen(R)
    g, u, dh = (normal(rng, R, I, dtype=dtype, scale=4.0) for _ in range(3))
    if R * I >= 64:
        g.view(-1)[:4] = torch.tensor([-100.0, 100.0, 0.0, -1.25], device="cuda").to(dtype)
    h, dg, du = bm.swiglu(g, u), *bm.swiglu_backward(dh, g, u)
    status_ok()
    wh, wg, wu = swiglu_ref(dh, g, u)
    gd, ud, dd = g.to(D), u.to(D), dh.to(D)
    s = torch.sigmoid(gd)
    # the fast exponential's error grows with its argument: |g| 2^-24 from its product with log2 e
    rel = (24 + 2 * gd.abs()) * 2.0 ** -24
    low = 2.0 ** -120  # sigma below the normal numbers may vanish
    check(h, wh, half_step(wh, dtype) + wh.abs() * rel + low, "h")
    check(du, wu, half_step(wu, dtype) + wu.abs() * rel + low, "du")
    check(dg, wg, half_step(wg, dtype) + (dd * ud).abs() * s * (1 + gd.abs()) * rel + low, "dg")


def test_swiglu_in_place_and_strided():
    rng = gen(3)
    R, I = 50, 128
    buf = normal(rng, R, 2 * I, dtype=F32)
    dh = normal(rng, R, I, dtype=F32)
    g, u = buf[:, :I], buf[:, I:]
    h = bm.swiglu(g, u)
    dg, du = bm.swiglu_backward(dh, g, u)
    keep = buf.clone()
    bm.swiglu_backward(dh, g, u, dg=g, du=u)
    assert torch.equal(buf[:, :I], dg) and torch.equal(buf[:, I:], du)
    buf.copy_(keep)
    assert bm.swiglu(g, u, out=u).data_ptr() == u.data_ptr()
    assert torch.equal(u, h) and torch.equal(g, keep[:, :I])
    status_ok()


def test_swiglu_gradient_against_differences():
    """Central differences in 64 bits of the kernel's own fp32 values: step 2^-7 (truncation below
    2^-14 / 6 times a third derivative of at most 1, rounding 2 x 2^-24 x 8 x 2^6)."""
    rng = gen(6)
    g, u, dh = (normal(rng, 16, 64, dtype=F32, scale=2.0) for _ in range(3))
    dg, du = bm.swiglu_backward(dh, g, u)
    e = 2.0 ** -7
    num_g = (bm.swiglu(g + e, u).to(D) - bm.swiglu(g - e, u).to(D)) / (2 * e) * dh.to(D)
    num_u = (bm.swiglu(g, u + e).to(D) - bm.swiglu(g, u - e).to(D)) / (2 * e) * dh.to(D)
    tol = dh.to(D).abs() * (u.to(D).abs() * 2.0 ** -14 + 64 * 12 * 2.0 ** -24 * (1 + g.to(D).abs() * u.to(D).abs()))
    check(dg, num_g, tol, "dg")
    check(du, num_u, tol + dh.to(D).abs() * 64 * 12 * 2.0 ** -24 * (1 + g.to(D).abs()), "du")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,I", [(1, 8), (77, 192), (40, 2560), (3, 20480)])
def test_swiglu_int8(R, I, dtype):
    """The codes are the quantiser's of SiLU(g) * u in FP32, but where that lies next to a code's edge."""
    rng = gen(I)
    g, u = normal(rng, R, I, dtype=dtype, scale=2.0), normal(rng, R, I, dtype=dtype)
    q, s = bm.swiglu_i8(g, u)
    status_ok()
    h = swiglu_ref(torch.zeros_like(g), g, u)[0]
    scale = h.abs().amax(dim=1) / 127
    assert ((s.to(D) - scale).abs() <= scale * 2.0 ** -18).all()
    # h within 64 roundings, the scale within 64: a code within half a step and 127 x 2^-17 of h / scale
    assert ((q.to(D) - h / scale[:, None]).abs() <= 0.5 + 127 * 2.0 ** -17).all()


def gates(R, I, dtype, across):
    """[R, I] gates: every 2^-8 from -130 to 130 and the type's largest of both signs; neighbours in a row, or
    (across) in a column, so that each row spans them all."""
    g = torch.arange(R * I, dtype=D, device="cuda") / 256 - 130
    g[-1], g[0] = torch.finfo(dtype).max, torch.finfo(dtype).min
    return (g.view(I, R).t() if across else g.view(R, I)).contiguous().to(dtype)


@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,I", [(260, 256), (13, 5120)])
def test_swiglu_of_every_gate(R, I, dtype, across):
    """Gates over the whole range of the exponential and past it: results are finite and the formula's.  A sigma
    below 2^-126 may be 0, so results are off by (1 + |g|) 2^-126 more (|u|, |dh| <= 1), and products of few
    2^-149 round to the subnormals."""
    rng = gen(I)
    g = gates(R, I, dtype, across)
    u, dh = ((torch.rand(R, I, generator=rng, device="cuda") * 2 - 1).to(dtype) for _ in range(2))
    h, dg, du = bm.swiglu(g, u), *bm.swiglu_backward(dh, g, u)
    status_ok()
    wh, wg, wu = swiglu_ref(dh, g, u)
    gd, ud, dd = g.to(D), u.to(D), dh.to(D)
    rel = (24 + 2 * gd.abs().clamp_max(130)) * 2.0 ** -24
    low = (1 + gd.abs().clamp_max(130)) * 2.0 ** -126 + 2.0 ** -146
    for t in (h, dg, du):
        assert t.isfinite().all()
    check(h, wh, half_step(wh, dtype) + wh.abs() * rel + low, "h")
    check(du, wu, half_step(wu, dtype) + wu.abs() * rel + low, "du")
    check(dg, wg, half_step(wg, dtype) + (dd * ud).abs() * torch.sigmoid(gd) * (1 + gd.abs()) * rel + low, "dg")


@pytest.mark.parametrize("across", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("R,I", [(260, 256), (13, 5120), (3, 22528)])
def test_swiglu_int8_of_every_gate(R, I, dtype, across):
    """The same gates through the quantiser: h within (24 + 2 x 130) 2^-24, the scale within that and three
    roundings more, so a code is within half a step and 127 times both; rows of vanishing h alone have scale 0."""
    rng = gen(I + 1)
    g = gates(R, I, dtype, across)
    u = (torch.rand(R, I, generator=rng, device="cuda") * 2 - 1).to(dtype)
    q, s = bm.swiglu_i8(g, u)
    status_ok()
    h = swiglu_ref(torch.zeros_like(g), g, u)[0]
    low, rel = 131 * 2.0 ** -126, 284 * 2.0 ** -24
    assert s.isfinite().all()
    check(s, h.abs().amax(dim=1) / 127, h.abs().amax(dim=1) / 127 * (rel + 3 * 2.0 ** -24) + low, "scale")
    step = s.to(D)[:, None]
    check(q.to(D) * step, h, step * (0.5 + 127 * (2 * rel + 4 * 2.0 ** -24)) + low, "codes")


# ---- together ---------------------------------------------------------------------------------------
def test_layer_training_step():
    """Router, dispatch, both first products, SwiGLU, second product and combine, then the experts'
    gradients: against autograd of the same layer in 64 bits on the kernel's routing."""
    T, H, I = 96, 256, 192
    cfg = bm.LayerConfig(hidden=H, inter=I, n_experts=16, n_groups=4, topk_groups=2, topk=4, group_topn=2)
    k, E = cfg.topk, cfg.n_experts
    g = gen(21)
    x, dy = normal(g, T, H), normal(g, T, H, scale=0.1)
    wr = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    wg, wu = normal(g, E, I, H, scale=H ** -0.5), normal(g, E, I, H, scale=H ** -0.5)
    wd = normal(g, E, H, I, scale=I ** -0.5)
    ids, w = bm.route(cfg, x, wr)
    p = bm.permute(cfg, ids)
    off = p["offsets"]
    rows = bm.gather_rows(cfg, x, p["dest_row"])
    gate, up = bm.grouped_mm(rows, wg, off), bm.grouped_mm(rows, wu, off)
    h = bm.swiglu(gate, up)
    o = bm.grouped_mm(h, wd, off, out_dtype=F32)
    y = bm.combine(cfg, o, p["dest_row"], w)
    # backward of the combine: each row gets its token's gradient times its weight
    token = (p["row_src"] // k).long()
    weight = w.view(-1)[p["row_src"].long()]
    do = (cfg.routed_scale * weight[:, None] * dy.float()[token]).to(BF)
    dh = bm.grouped_mm_dgrad(do, wd, off)
    dwd = bm.grouped_mm_wgrad(do, h, off, out_dtype=F32)
    dgate, dup = bm.swiglu_backward(dh, gate, up)
    dwg = bm.grouped_mm_wgrad(dgate, rows, off, out_dtype=F32)
    dwu = bm.grouped_mm_wgrad(dup, rows, off, out_dtype=F32)
    drows = bm.grouped_mm_dgrad(dgate, wg, off, out_dtype=F32) + bm.grouped_mm_dgrad(dup, wu, off, out_dtype=F32)
    dx = torch.zeros(T, H, device="cuda").index_add_(0, token, drows)
    status_ok()

    leaves = [t.to(D).requires_grad_() for t in (x, wg, wu, wd)]
    X, G, U, Dn = leaves
    out = torch.zeros(T, H, dtype=D, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            a = G[e] @ X[t]
            out[t] = out[t] + cfg.routed_scale * w[t, j].to(D) * (Dn[e] @ (a * torch.sigmoid(a) * (U[e] @ X[t])))
    out.backward(dy.to(D))
    # gate, up, h, do, dh, dgate and dup are each rounded to bf16 once (2^-9 of a value, relative to norms):
    # at most seven such roundings lie on a gradient's path
    for name, got, want in (("y", y, out), ("dx", dx, X.grad), ("dw_gate", dwg, G.grad), ("dw_up", dwu, U.grad),
                            ("dw_down", dwd, Dn.grad)):
        rel = ((got.to(D) - want).norm() / want.norm()).item()
        assert rel <= 8 * 2.0 ** -8, (name, rel)
    ref = bm.forward(cfg, x, wr, None, wg, wu, wd)
    assert ((y.to(D) - ref.to(D)).norm() / ref.to(D).norm()).item() <= 8 * 2.0 ** -8


def test_int8_experts_together():
    """Quantise, both first products, SwiGLU with quantisation, second product: against the same steps in
    64 bits on the kernel's codes at each step's input."""
    E, R, H, I = 6, 200, 256, 192
    g = gen(31)
    counts = ragged_counts(E, R, 9)
    off = offsets_of(counts)
    x = normal(g, R, H)
    q8 = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    wg, wu, wd = q8(E, I, H), q8(E, I, H), q8(E, H, I)
    sg, su, sd = (torch.rand(E, n, generator=g, device="cuda") / 1000 + 1e-4 for n in (I, I, H))
    q, s = bm.quant_i8_rows(x)
    gate = bm.grouped_mm_i8(q, s, wg, sg, off, out_dtype=F32)
    up = bm.grouped_mm_i8(q, s, wu, su, off, out_dtype=F32)
    hq, hs = bm.swiglu_i8(gate, up)
    y = bm.grouped_mm_i8(hq, hs, wd, sd, off)
    status_ok()
    h = swiglu_ref(torch.zeros_like(gate), gate, up)[0]
    assert ((hq.to(D) * hs.to(D)[:, None] - h).abs() <= hs.to(D)[:, None] * (0.5 + 127 * 2.0 ** -16)).all()
    for e, a, b in spans(counts):
        want = (q[a:b].to(D) @ wg[e].to(D).t()) * s[a:b].to(D)[:, None] * sg[e].to(D)
        check(gate[a:b], want, want.abs() * (4 * 2.0 ** -24), "gate")
        want = (hq[a:b].to(D) @ wd[e].to(D).t()) * hs[a:b].to(D)[:, None] * sd[e].to(D)
        check(y[a:b], want, half_step(want, BF) + want.abs() * (4 * 2.0 ** -24), "y")


def test_captured_and_replayed_with_other_groups():
    """A graph of the products reads offsets and inputs at replay; two graphs do not share anything."""
    E, R, K, N = 8, 512, 256, 192
    g = gen(41)
    w = normal(g, E, N, K, scale=K ** -0.5)
    x, dy = normal(g, R, K), normal(g, R, N)
    off = offsets_of(ragged_counts(E, R, 1))
    run_all(x, dy, w, off, BF)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run_all(x, dy, w, off, BF))
        graphs.append(graph)
    for seed in (2, 3):
        counts = ragged_counts(E, R, seed)
        off.copy_(offsets_of(counts))
        x.copy_(normal(g, R, K))
        want = run_all(x, dy, w, off, BF)
        for graph, got in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(got[k], want[k]) for k in want)
    status_ok()


@pytest.mark.parametrize("R,E", [(1, 1), (40, 8), (700, 8), (9000, 2)])
def test_calls_that_follow_one_another(R, E):
    """Calls back to back over the same buffers, with other work of the stream between them, eager and captured: each
    sees what the one before it wrote, and nothing is written before its last reader is done."""
    I, H, n = 320, 512, 12
    g = gen(R)
    off = offsets_of(ragged_counts(E, R, 4, empty=0.0))
    q8, _, w8, cs = i8_operands(g, E, R, H, I)
    w, down = normal(g, E, I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    x, steps = torch.empty(R, H, dtype=BF, device="cuda"), normal(g, n, R, H)
    q, s = torch.empty_like(q8), torch.empty(R, device="cuda")
    a, b, h = (torch.empty(R, I, dtype=BF, device="cuda") for _ in range(3))
    dx, dw = torch.empty_like(x), torch.zeros(E, H, I, device="cuda")
    out = torch.empty(n, 2, R, H, dtype=BF, device="cuda")

    def run(sync):
        dw.zero_()
        for i in range(n):
            calls = (lambda: x.copy_(steps[i]), lambda: bm.quant_i8_rows(x, q, s),
                     lambda: bm.grouped_mm_i8(q, s, w8, cs, off, out=a), lambda: bm.grouped_mm(x, w, off, out=b),
                     lambda: bm.swiglu(b, b, out=h), lambda: bm.grouped_mm(h, down, off, out=out[i, 0]),
                     lambda: bm.swiglu_backward(a, b, h, dg=a, du=b), lambda: bm.grouped_mm_dgrad(a, w, off, out=dx),
                     lambda: bm.grouped_mm_wgrad(dx, b, off, out=dw, accumulate=True), lambda: out[i, 1].copy_(dx))
            for f in calls:
                f()
                if sync:
                    torch.cuda.synchronize()
        return out.clone(), dw.clone()

    want = run(True)
    got = [run(False) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(False)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        got.append(tuple(t.clone() for t in captured))
    status_ok()
    for result in got:
        assert all(torch.equal(r.nan_to_num(), v.nan_to_num()) for r, v in zip(result, want))


@pytest.mark.parametrize("R,E", [(1, 1), (40, 8), (700, 8)])
def test_int8_calls_that_follow_one_another(R, E):
    """Quantisers and products back to back over the same buffers: finite, and bit for bit what they give with a wait
    behind each call."""
    H, I, n = 512, 320, 16
    g = gen(R + 7)
    off = offsets_of(ragged_counts(E, R, 6, empty=0.0))
    w8 = [torch.randint(-127, 128, (E, a, b), generator=g, device="cuda", dtype=torch.int8)
          for a, b in ((I, H), (I, H), (H, I))]
    cs = [torch.rand(E, a, generator=g, device="cuda") / 1000 + 1e-4 for a in (I, I, H)]
    x, steps = torch.empty(R, H, dtype=BF, device="cuda"), normal(g, n, R, H)
    q, s, hq, hs = bm.quant_i8_rows(steps[0]) + (torch.empty(R, I, dtype=torch.int8, device="cuda"),
                                                 torch.empty(R, device="cuda"))
    gate, up = (torch.empty(R, I, device="cuda") for _ in range(2))
    out = torch.empty(n, R, H, device="cuda")

    def run(sync):
        out.zero_()
        for i in range(n):
            for f in (lambda: x.copy_(steps[i]), lambda: bm.quant_i8_rows(x, q, s),
                      lambda: bm.grouped_mm_i8(q, s, w8[0], cs[0], off, out=gate),
                      lambda: bm.grouped_mm_i8(q, s, w8[1], cs[1], off, out=up),
                      lambda: bm.swiglu_i8(gate, up, hq, hs),
                      lambda: bm.grouped_mm_i8(hq, hs, w8[2], cs[2], off, out=out[i])):
                f()
                if sync:
                    torch.cuda.synchronize()
        return out.clone()

    want = run(True)
    assert want.isfinite().all() and (want != 0).any(dim=2).all()
    for _ in range(4):
        assert torch.equal(run(False), want)
    status_ok()


def test_two_calls_at_once():
    """Products of different kernels on two streams, overlapping: each gives what it gives alone."""
    g = gen(61)
    big = (normal(g, 9000, 1024), normal(g, 9000, 2048), normal(g, 4, 2048, 1024), offsets_of([3000, 1, 0, 5999]))
    few = (normal(g, 40, 2048), normal(g, 40, 512), normal(g, 16, 512, 2048), offsets_of(ragged_counts(16, 40, 5)))
    want = [run_all(*a, BF) for a in (big, few)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, a in enumerate((big, few)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run_all(*a, BF))
    status_ok()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(r[k], want[i][k]) for k in r)


def test_results_past_32_bits():
    """Outputs of more than 2^31 elements: their first and last rows, and the last expert's gradient."""
    g = gen(71)
    R, K, N = 270000, 64, 8192
    x, w = normal(g, R, K), normal(g, N, K, scale=K ** -0.5)
    out = bm.grouped_mm(x, w)
    assert out.numel() > 2 ** 31
    for a in (slice(0, 300), slice(R - 300, R)):
        v = x[a].to(D) @ w.to(D).t()
        check(out[a], v, half_step(v, BF) + sum_tol(x[a].to(D).abs() @ w.to(D).abs().t(), K, BF), "out")
    del out
    counts = [2] * 255 + [90]
    dy, x = normal(g, sum(counts), 4096), normal(g, sum(counts), 4096)
    dw = bm.grouped_mm_wgrad(dy, x, offsets_of(counts))
    assert dw.numel() > 2 ** 31
    for e, a, b in ((0, 0, 2), (255, 510, 600)):
        v = dy[a:b].to(D).t() @ x[a:b].to(D)
        check(dw[e], v, half_step(v, BF) + sum_tol(dy[a:b].to(D).abs().t() @ x[a:b].to(D).abs(), b - a, BF), f"dw {e}")
    status_ok()


def test_binding_refusals():
    x, w = normal(gen(1), 6, 64), normal(gen(2), 2, 32, 64)
    off = offsets_of([2, 4])
    for f in (lambda: bm.grouped_mm(x, w),                                   # two experts need offsets
              lambda: bm.grouped_mm(x, w, offsets_of([1, 2, 3])),            # offsets of three
              lambda: bm.grouped_mm(x[:, :32], w, off),                      # widths differ
              lambda: bm.grouped_mm(x.t(), w, off),                          # columns, not rows, contiguous
              lambda: bm.grouped_mm(x[:1].expand(6, 64), w, off),            # one row over and over
              lambda: bm.grouped_mm(x, w.transpose(0, 1), off),              # weights not packed
              lambda: bm.grouped_mm(x, w, off, out=torch.empty(5, 32, dtype=BF, device="cuda")),
              lambda: bm.grouped_mm_wgrad(x, x[:5], off),
              lambda: bm.grouped_mm_wgrad(x, x, off[:1]),
              lambda: bm.grouped_mm_wgrad(x, x, off, out=torch.empty(2, 64, 32, dtype=BF, device="cuda")),
              lambda: bm.grouped_mm_wgrad(x, x, off, accumulate=True),
              lambda: bm.swiglu(x, x[:5])):
        with pytest.raises(ValueError):
            f()
    one = torch.ones(2, 32, device="cuda")
    q, s = bm.quant_i8_rows(x)
    for f in (lambda: bm.grouped_mm_i8(q, None, w.to(torch.int8), one, off),
              lambda: bm.grouped_mm_i8(q, s, w.to(torch.int8), None, off), lambda: bm.grouped_mm(x, None, off),
              lambda: bm.grouped_mm_wgrad(x, x, [0, 2, 6]), lambda: bm.swiglu(x, None),
              lambda: bm.grouped_mm(x, w.to(HF), off), lambda: bm.grouped_mm(x.float(), w.float(), off),
              lambda: bm.grouped_mm(x, w, off.int()), lambda: bm.grouped_mm(x, w, off, out_dtype=torch.int8),
              lambda: bm.grouped_mm(x, w, off, out=torch.empty(6, 32, device="cuda"), out_dtype=BF),
              lambda: bm.swiglu(x, x.float())):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: bm.grouped_mm(x, w, off, out_dtype=HF),
              lambda: bm.grouped_mm(normal(gen(1), 6, 65)[:, 1:], w, off),   # rows off the 16-byte boundaries
              lambda: bm.grouped_mm_wgrad(x, x, off, out=torch.zeros(2, 64, 64, dtype=BF, device="cuda"),
                                          accumulate=True)):
        with pytest.raises(bm.BeamMoeError):
            f()
    status_ok()


def test_on_another_stream():
    g = gen(51)
    E, R, K, N = 1, 20000, 128, 64  # the weight gradient takes a workspace here
    x, dy, w = normal(g, R, K), normal(g, R, N), normal(g, E, N, K)
    want = run_all(x, dy, w, None, BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dict(out=bm.grouped_mm(x, w, stream=side), dx=bm.grouped_mm_dgrad(dy, w, stream=side),
               dw=bm.grouped_mm_wgrad(dy, x, stream=side))
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    # by its handle; what a call returns belongs to that stream, whose later work may use it unordered
    got = dict(out=bm.grouped_mm(x, w, stream=side.cuda_stream), dx=bm.grouped_mm_dgrad(dy, w, stream=side.cuda_stream),
               dw=bm.grouped_mm_wgrad(dy, x, stream=side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    status_ok()


def test_results_are_detached():
    """Inputs that require gradients are taken; what comes back does not claim to have any."""
    g = gen(81)
    x, w = normal(g, 40, 64).requires_grad_(), normal(g, 32, 64).requires_grad_()
    out = bm.grouped_mm(x, w)
    h = bm.swiglu(out, out)
    q, s = bm.quant_i8_rows(x)
    for t in (out, h, s, bm.grouped_mm_dgrad(out, w), bm.grouped_mm_wgrad(out, x), *bm.swiglu_backward(h, out, out)):
        assert not t.requires_grad and t.isfinite().all()
    status_ok()
