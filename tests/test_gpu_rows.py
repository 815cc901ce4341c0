"""GPU parity of the row operators (tokens sorted by expert and back, their gradients, e4m3
quantising, the grouped e4m3 product) against the float64 oracle, through the binding.

Tolerances.  u = 2^-24.  Rows that are only moved, and gates of one slot, must be equal.  A sum of
n fp32 terms taken in any order is off by at most n u sum|term|, a rounding to type t by half of
eps(t) of the value.  Quantised rows are equal bit for bit (the definition fixes every rounding).
The product's sums are checked twice: with integers whose sums fp32 holds exactly (equality), and
with ordinary values.  For fp32 results each addition inside a block may lose up to 2u of the
running sum (a matrix instruction may truncate), so 2 (K + blocks + 4) u sum|term|.  For 16-bit
results the e4m3 matrix instruction brings its 128 products to the exponent of the largest and
keeps what is at least 2^-13 of it (seen with powers of two: a second product of 2^-13 of the
first is kept, one of 2^-14 is lost), so each product may lose 2^-13 of the block's largest, a
block 128 2^-13 = 2^-6 of it.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
import any_precision_expert_router_amd as apq  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SMALLEST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}   # half a subnormal step


def say(*a):
    print(*a, flush=True)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(DEV) if dtype is None else t.to(DEV, dtype)


def f64(t):
    return t.double().cpu().numpy()


class Routing:
    """ids [T, k] with some naming no expert, grouped by the library."""

    def __init__(self, T, E, k, seed, drop=0.0, repeat=False):
        r = np.random.default_rng(seed)
        if repeat:
            ids = r.integers(0, E, size=(T, k))            # one expert in several slots
        else:
            ids = np.argsort(r.random((T, E)), axis=1)[:, :k]
        bad = r.random((T, k)) < drop
        ids = np.where(bad, np.where(r.random((T, k)) < 0.5, -1, E + 3), ids).astype(np.int32)
        self.T, self.E, self.k, self.ids = T, E, k, dev(ids)
        self.gates = dev(r.random((T, k)).astype(np.float32) + 0.01)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        self.pairs = torch.full((max(T * k, 1),), -7, dtype=torch.int32, device=DEV)
        active = torch.empty(E, dtype=torch.int32, device=DEV)
        apq.moe_group_by_expert(self.ids, E, self.offsets, self.pairs, active, torch.empty(1, dtype=torch.int32, device=DEV))
        self.pairs = self.pairs[:T * k]
        off, pairs, _, _ = oracle.group_by_expert(ids, E)
        self.off = np.asarray(off)
        self.n = int(self.off[-1])
        self.pairs_np = np.asarray(pairs)[:self.n]
        np.testing.assert_array_equal(self.offsets.cpu().numpy(), self.off)
        np.testing.assert_array_equal(self.pairs.cpu().numpy()[:self.n], self.pairs_np)
        self.rows_np = oracle.pair_rows(self.pairs_np, self.n, T * k).reshape(T, k)
        self.rows = dev(self.rows_np)
        self.groups = [range(int(self.off[e]), int(self.off[e + 1])) for e in range(E)]


def strided(rows, cols, dtype, fill, extra):
    """A [rows, cols] view with `extra` more elements between rows, all memory holding `fill`."""
    return torch.full((rows, cols + extra), fill, dtype=dtype, device=DEV)[:, :cols]


MOVE_CASES = [  # T, E, k, H, type, extra stride, dropped share, repeated experts
    (1, 1, 1, 1, "f16", 0, 0.0, False),
    (1, 8, 2, 4096, "f16", 0, 0.0, False),
    (16, 60, 4, 2048, "f16", 0, 0.0, False),
    (5, 8, 3, 131, "bf16", 0, 0.0, False),
    (7, 4, 2, 8, "f32", 3, 0.3, False),
    (33, 64, 8, 517, "f16", 1, 0.3, False),
    (9, 16, 10, 1025, "f32", 0, 0.2, True),
    (3, 1024, 32, 64, "bf16", 8, 0.0, False),
    (130, 512, 10, 2050, "bf16", 5, 0.05, False),
    (300, 3, 2, 777, "f16", 0, 0.0, True),
    (700, 64, 8, 1000, "bf16", 0, 0.1, False),
    (4, 8, 2, 20001, "f32", 0, 0.0, False),
    (6, 8, 4, 256, "f16", 0, 1.0, False),     # no pair names an expert
]


@pytest.mark.parametrize("T,E,k,H,ty,extra,drop,repeat", MOVE_CASES)
def test_permute_and_its_gradient(T, E, k, H, ty, extra, drop, repeat):
    say(f"permute T={T} E={E} k={k} H={H} {ty} extra={extra} drop={drop}")
    dt, r = TYPES[ty], Routing(T, E, k, T + H, drop, repeat)
    g = torch.Generator(device=DEV).manual_seed(H)
    x = strided(T, H, dt, float("nan"), extra)
    x.copy_(torch.randn(T, H, device=DEV, generator=g))
    xs = strided(T * k, H, dt, 5.0, extra)
    rows = torch.full((T, k), 99, dtype=torch.int32, device=DEV)
    apq.moe_permute_tokens(x, r.ids, r.offsets, r.pairs, xs, rows)
    np.testing.assert_array_equal(rows.cpu().numpy(), r.rows_np)
    assert torch.equal(xs[:r.n], x[dev(r.pairs_np // k).long()])
    assert bool((xs[r.n:] == 5.0).all())
    if extra:
        assert bool((xs.as_strided((T * k, extra), (H + extra, 1), H) == 5.0).all())

    dxs = strided(T * k, H, dt, float("nan"), extra)     # rows behind the last group stay NaN: never read
    dxs[:r.n] = torch.randn(r.n, H, device=DEV, generator=g)
    dx = strided(T, H, dt, 7.0, extra)
    apq.moe_permute_tokens_backward(dxs, r.rows, dx)
    want, size = oracle.unpermute_tokens(f64(dxs), r.rows_np)
    err = np.abs(f64(dx) - want)
    assert (err <= HALF[ty] * np.abs(want) * (1 + 2 * k * U) + k * U * size + SMALLEST[ty]).all()
    if extra:
        assert bool((dx.as_strided((T, extra), (H + extra, 1), H) == 7.0).all())


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,E,k,H,ty,extra,drop,repeat", MOVE_CASES)
def test_unpermute_and_its_gradient(T, E, k, H, ty, extra, drop, repeat, gated):
    say(f"unpermute T={T} E={E} k={k} H={H} {ty} extra={extra} drop={drop} gated={gated}")
    dt, r = TYPES[ty], Routing(T, E, k, T + H + 1, drop, repeat)
    g = torch.Generator(device=DEV).manual_seed(H + 1)
    ys = strided(T * k, H, dt, float("nan"), extra)
    ys[:r.n] = torch.randn(r.n, H, device=DEV, generator=g)
    add = strided(T, H, dt, float("nan"), extra)
    add.copy_(torch.randn(T, H, device=DEV, generator=g))
    gates = r.gates.clone()
    gates[r.rows < 0] = float("nan")                     # a pair without a row contributes nothing
    gates_np = f64(gates) if gated else None
    for residual in (None, add):
        y = strided(T, H, dt, 7.0, extra)
        apq.moe_unpermute_tokens(ys, r.rows, gates if gated else None, y, add=residual)
        want, size = oracle.unpermute_tokens(f64(ys), r.rows_np, gates_np, None if residual is None else f64(add))
        err = np.abs(f64(y) - want)
        assert (err <= HALF[ty] * np.abs(want) * (1 + 2 * k * U) + (k + 2) * U * size + SMALLEST[ty]).all()

    dy = strided(T, H, dt, float("nan"), extra)
    dy.copy_(torch.randn(T, H, device=DEV, generator=g))
    dys = strided(T * k, H, dt, 5.0, extra)
    dgates = torch.full((T, k), 9.0, device=DEV)
    apq.moe_unpermute_tokens_backward(dy, ys, r.rows, gates if gated else None, dys, dgates)
    want_dys, want_dg, size = oracle.unpermute_tokens_grad(f64(dy), f64(ys), r.rows_np, gates_np)
    got = f64(dys)
    for row, want in want_dys.items():
        assert (np.abs(got[row] - want) <= HALF[ty] * np.abs(want) * (1 + 2 * U) + U * np.abs(want) + SMALLEST[ty]).all()
    assert (got[r.n:] == 5.0).all()
    assert (np.abs(f64(dgates) - want_dg) <= (H + 2) * U * size).all()
    # each output alone
    dys2, dg2 = torch.full_like(dys, 5.0), torch.full_like(dgates, 3.0)
    apq.moe_unpermute_tokens_backward(dy, None, r.rows, gates if gated else None, dys2, None)
    apq.moe_unpermute_tokens_backward(dy, ys, r.rows, gates if gated else None, None, dg2)
    assert torch.equal(dys2, dys) and torch.equal(dg2, dgates)


def test_gradients_against_differences():
    """d/dgates and d/dx of L = <unpermute(2 permute(x), gates), c> against central differences: L is
    linear in each, so differences are exact up to the fp32 roundings of the two outputs."""
    T, E, k, H = 6, 5, 3, 40
    r = Routing(T, E, k, 3, drop=0.2)
    rng = np.random.default_rng(4)
    x, c = dev(rng.standard_normal((T, H)).astype(np.float32)), dev(rng.standard_normal((T, H)).astype(np.float32))

    def forward(x, gates):
        xs, rows = torch.zeros(T * k, H, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
        apq.moe_permute_tokens(x, r.ids, r.offsets, r.pairs, xs, rows)
        ys, y = 2 * xs, torch.empty(T, H, device=DEV)
        apq.moe_unpermute_tokens(ys, rows, gates, y)
        return y, ys, rows

    def loss(x, gates):
        return float((forward(x, gates)[0].double() * c.double()).sum())

    y, ys, rows = forward(x, r.gates)
    dys, dgates = torch.zeros_like(ys), torch.empty(T, k, device=DEV)
    apq.moe_unpermute_tokens_backward(c, ys, rows, r.gates, dys, dgates)
    dx = torch.empty_like(x)
    apq.moe_permute_tokens_backward(2 * dys, rows, dx)
    h = 0.5
    scale = float(c.abs().double().sum()) * float(ys.abs().max()) * k * 4      # bounds sum |c y| for every shift
    tol = 8 * U * scale / h
    for t in range(T):
        for j in range(k):
            up, down = r.gates.clone(), r.gates.clone()
            up[t, j] += h
            down[t, j] -= h
            d = (loss(x, up) - loss(x, down)) / float(up[t, j].double() - down[t, j].double())
            assert abs(d - float(dgates[t, j])) <= tol
    for t, col in [(0, 0), (3, 17), (5, 39)]:
        up, down = x.clone(), x.clone()
        up[t, col] += h
        down[t, col] -= h
        d = (loss(up, r.gates) - loss(down, r.gates)) / float(up[t, col].double() - down[t, col].double())
        assert abs(d - float(dx[t, col])) <= tol


QUANT_CASES = [  # M, K, type, extra stride, valid rows (None: all)
    (1, 1, "f16", 0, None), (1, 128, "bf16", 0, None), (3, 127, "f32", 0, None), (16, 2048, "f16", 0, None),
    (5, 129, "bf16", 3, None), (40, 1000, "f16", 1, 17), (130, 2560, "bf16", 0, 0), (64, 511, "f32", 2, 63),
    (9, 513, "f16", 0, None), (300, 3584, "bf16", 0, 299), (2, 40, "f32", 0, 5),
]


def _limit(rows, M):
    return (None, M) if rows is None else (dev(np.array([rows], dtype=np.int32)), min(rows, M))


@pytest.mark.parametrize("M,K,ty,extra,rows", QUANT_CASES)
def test_quantize_bit_exact(M, K, ty, extra, rows):
    say(f"quantize M={M} K={K} {ty} extra={extra} rows={rows}")
    g = torch.Generator(device=DEV).manual_seed(M * K)
    x = strided(M, K, TYPES[ty], float("nan"), extra)
    x.copy_(torch.randn(M, K, device=DEV, generator=g) * torch.exp(3 * torch.randn(M, 1, device=DEV, generator=g)))
    if M > 2:
        x[1] = 0
        x[2, ::3] = 0
    q = strided(M, K, torch.uint8, 77, extra)
    scales = torch.full((M, -(-K // 128)), -1.0, device=DEV)
    n_rows, n = _limit(rows, M)
    apq.moe_fp8_quantize(x, q, scales, n_rows=n_rows)
    codes, want = oracle.fp8_quantize(x.float().cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy()[:n], want[:n])
    np.testing.assert_array_equal(q.cpu().numpy()[:n], codes[:n])
    assert bool((scales[n:] == -1).all()) and bool((q[n:] == 77).all())
    if extra:
        assert bool((q.as_strided((M, extra), (K + extra, 1), K) == 77).all())


def test_quantize_of_extreme_values():
    """Infinities and NaN become NaN and leave their block alone; tiny, huge and subnormal blocks."""
    x = torch.zeros(8, 256, device=DEV)
    x[0] = 3.0
    x[0, 5], x[0, 9], x[0, 200] = float("inf"), float("nan"), float("-inf")
    x[1, :128] = float("nan")
    x[2] = 2.0 ** -120
    x[3] = 3.4e38
    x[3, ::2] = -1e30
    x[4] = 2.0 ** -140
    x[5, 0] = 2.0 ** -100
    x[6] = torch.linspace(-1, 1, 256, device=DEV)
    x[7] = -0.0
    q, scales = torch.empty(8, 256, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(8, 2, device=DEV)
    apq.moe_fp8_quantize(x, q, scales)
    codes, want = oracle.fp8_quantize(x.cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy(), want)
    got = q.view(torch.uint8).cpu().numpy()
    nan = (codes & 127) == 127
    np.testing.assert_array_equal((got & 127) == 127, nan)
    np.testing.assert_array_equal(got[~nan], codes[~nan])


@pytest.mark.parametrize("M,K,ty,extra,rows", QUANT_CASES)
def test_quantize_silu(M, K, ty, extra, rows):
    """The gate costs at most 4 ulp (exp 1, its correction and 1 + e half each, rcp 1, two products
    half each), e4m3 half a step of 3 fraction bits (or of its smallest step)."""
    say(f"quantize_silu M={M} K={K} {ty} extra={extra} rows={rows}")
    g = torch.Generator(device=DEV).manual_seed(M * K + 1)
    x = strided(M, 2 * K, TYPES[ty], float("nan"), extra)
    x.copy_(torch.randn(M, 2 * K, device=DEV, generator=g) * torch.exp(2 * torch.randn(M, 1, device=DEV, generator=g)))
    q = strided(M, K, torch.uint8, 77, extra)
    scales = torch.full((M, -(-K // 128)), -1.0, device=DEV)
    n_rows, n = _limit(rows, M)
    apq.moe_fp8_quantize_silu(x, q, scales, n_rows=n_rows)
    v = f64(x)
    v = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    for r in range(n):
        for b in range(scales.shape[1]):
            block = v[r, b * 128:(b + 1) * 128]
            m = max(np.abs(block).max(), 2.0 ** -100)
            s = float(scales[r, b])
            assert abs(s - m / 448) <= 10 * U * m / 448
            got = oracle.e4m3_values()[q[r, b * 128:b * 128 + len(block)].cpu().numpy()] * s
            assert (np.abs(got - block) <= np.maximum(2.0 ** -4 * np.abs(block), 2.0 ** -10 * s) * (1 + 32 * U)
                    + 12 * U * np.abs(block)).all()
    assert bool((scales[n:] == -1).all()) and bool((q[n:] == 77).all())


def test_quantize_silu_far_gates():
    """Gates where exp over- or underflows: silu(z) is z or 0 there, never NaN."""
    z = np.array([-3e38, -1e4, -200, -104, -89, -88, -87.3, -20, 0, 20, 87, 89, 200, 1e4, 3e38], dtype=np.float32)
    x = torch.zeros(len(z), 2, device=DEV)
    x[:, 0], x[:, 1] = dev(z), 1.0
    q, scales = torch.empty(len(z), 1, dtype=torch.uint8, device=DEV), torch.empty(len(z), 1, device=DEV)
    apq.moe_fp8_quantize_silu(x, q, scales)
    with np.errstate(over="ignore"):
        want = z.astype(np.float64) / (1 + np.exp(-z.astype(np.float64)))
    m = np.maximum(np.abs(want), 2.0 ** -100) / 448
    assert (np.abs(f64(scales)[:, 0] - m) <= 10 * U * m).all()


# ------------------------------------------------------------------------------------------
# the product
# ------------------------------------------------------------------------------------------
GEMM_CASES = [  # T, E, k, N, K, type, gather, dropped share, repeated experts
    (1, 1, 1, 1, 16, "f32", False, 0.0, False),
    (1, 8, 2, 64, 128, "f32", True, 0.0, False),
    (1, 8, 2, 96, 4096, "f16", True, 0.0, False),
    (4, 8, 2, 33, 144, "f32", True, 0.0, False),
    (16, 60, 4, 130, 640, "bf16", True, 0.0, False),
    (17, 3, 2, 129, 272, "f32", False, 0.3, False),
    (33, 64, 8, 257, 512, "f32", True, 0.2, False),
    (64, 4, 2, 160, 384, "bf16", False, 0.0, False),
    (100, 2, 2, 300, 1040, "f16", True, 0.1, False),
    (150, 1, 1, 260, 256, "f32", False, 0.0, False),
    (257, 1, 1, 515, 400, "f32", False, 0.0, False),
    (300, 5, 3, 384, 896, "bf16", True, 0.05, True),
    (520, 2, 1, 520, 1152, "f32", True, 0.0, False),
    (1000, 200, 4, 144, 256, "f32", True, 0.02, False),
    (90, 1024, 10, 40, 128, "f32", True, 0.0, False),
    (3000, 2, 2, 272, 128, "f32", False, 0.0, False),
    (8, 8, 4, 64, 256, "f32", True, 1.0, False),
]


def _gemm_inputs(r, N, K, gather, integers, seed):
    rng = np.random.default_rng(seed)
    R, kb, nb = (r.T if gather else r.T * r.k), -(-K // 128), -(-N // 128)
    if integers:      # sums of up to K 64 * 16 quarter units: exact in fp32 for K <= 4096
        table = oracle.e4m3_values()
        small = np.array([c for c in range(256) if abs(table[c]) <= 8 and table[c] == np.rint(table[c])], dtype=np.uint8)
        a, w = rng.choice(small, size=(R, K)), rng.choice(small, size=(r.E, N, K))
        sa = rng.choice([0.5, 1.0, 2.0], size=(R, kb)).astype(np.float32)
        sw = rng.choice([0.5, 1.0, 2.0], size=(r.E, nb, kb)).astype(np.float32)
    else:
        a = oracle.e4m3_encode(np.clip(rng.standard_normal((R, K)) * 120, -448, 448))
        w = oracle.e4m3_encode(np.clip(rng.standard_normal((r.E, N, K)) * 120, -448, 448))
        sa = (np.exp(rng.standard_normal((R, kb))) / 120).astype(np.float32)
        sw = (np.exp(rng.standard_normal((r.E, nb, kb))) / 2400).astype(np.float32)
    return a, sa, w, sw


def _gemm(r, a, sa, w, sw, ty, gather, N, extra=3, grouped=True):
    """c through the library, from rows of a with NaN between and behind them."""
    R, K = a.shape
    padded = torch.full((R, (K + 15) // 16 * 16 + 16), 127, dtype=torch.uint8, device=DEV)   # 127: NaN
    at = padded[:, :K]
    at.copy_(dev(a))
    c = strided(r.T * r.k, N, TYPES[ty], 55.0, extra)
    apq.moe_fp8_gemm(at, dev(sa), dev(w) if grouped else dev(w[0]), dev(sw), c,
                     expert_offsets=r.offsets if grouped else None, sorted_pairs=r.pairs if gather else None, k=r.k)
    assert bool((c[r.n:] == 55.0).all())
    assert bool((c.as_strided((c.shape[0], extra), (N + extra, 1), N) == 55.0).all())
    return c


def _worst(got, want, size, top, K, ty):
    """The largest error over its bound."""
    tol = 2 * (K + -(-K // 128) + 4) * U * size + HALF[ty] * np.abs(want) * (1 + K * U) + SMALLEST[ty]
    if ty != "f32":
        tol += 2.0 ** -6 * (1 + HALF[ty]) * top
    return float((np.abs(got - want) / tol).max(initial=0))


@pytest.mark.parametrize("integers", [True, False], ids=["integers", "values"])
@pytest.mark.parametrize("T,E,k,N,K,ty,gather,drop,repeat", GEMM_CASES)
def test_gemm(T, E, k, N, K, ty, gather, drop, repeat, integers):
    say(f"gemm T={T} E={E} k={k} N={N} K={K} {ty} gather={gather} drop={drop} integers={integers}")
    r = Routing(T, E, k, T + N, drop, repeat)
    a, sa, w, sw = _gemm_inputs(r, N, K, gather, integers, T * 3 + K)
    source = r.pairs_np // k if gather else np.arange(T * k)
    want, size, top = oracle.fp8_gemm(a, sa, w, sw, r.groups, source)
    ways = [True] if E > 1 or drop else [True, False]
    for grouped in ways:
        c = _gemm(r, a, sa, w, sw, ty, gather, N, grouped=grouped)[:r.n]
        if integers:
            exact = torch.from_numpy(want[:r.n]).to(TYPES[ty])
            assert torch.equal(c.cpu(), exact)
        else:
            assert _worst(f64(c), want[:r.n], size[:r.n], top[:r.n], K, ty) <= 1


# Sizes that fill the chip, so that each form of the product runs: tiles of few rows, tiles of many (of
# every height), several tiles to a workgroup, more blocks of K than their scales are staged for, a
# short last block behind them.  The reference is torch's float64 product on the device.
BIG_GEMM_CASES = [  # T, E, k, N, K, type, gather, dropped share
    (64, 64, 2, 2100, 528, "bf16", True, 0.0),       # few rows each, 576 tiles
    (96, 8, 2, 16400, 3728, "f16", True, 0.1),       # 24 rows each, 29 whole blocks and a short one
    (96, 8, 2, 16400, 400, "f32", False, 0.0),
    (600, 2, 1, 8200, 400, "bf16", True, 0.0),       # about 300 rows each: two tiles of up to 160
    (600, 2, 1, 8200, 400, "f32", True, 0.05),
    (520, 1, 1, 8200, 3728, "bf16", False, 0.0),
    (520, 1, 1, 8200, 3728, "f32", False, 0.0),
    (1500, 6, 1, 5130, 128, "f16", True, 0.0),       # one block only; about 250 rows each
    (700, 40, 2, 4100, 64, "bf16", False, 0.02),     # no whole block
    (1900, 40, 3, 2050, 272, "bf16", True, 0.0),
    (256, 1, 1, 4100, 640, "bf16", False, 0.0),      # 128 tiles of few rows
    (1, 1, 1, 4100, 2064, "bf16", False, 0.0),       # 16-column tiles
    (40, 1, 1, 4100, 528, "f32", False, 0.0),        # 32-row stream
] + [(n, 1, 1, 8300, 272, "bf16", False, 0.0) for n in (64, 145, 257)] + [
    (16 * n, 16, 1, 8200, 272, ty, True, 0.0) for n in (40, 70, 100, 125, 150, 180, 210, 245) for ty in ("bf16", "f32")]


@pytest.mark.parametrize("T,E,k,N,K,ty,gather,drop", BIG_GEMM_CASES)
def test_gemm_on_the_whole_chip(T, E, k, N, K, ty, gather, drop):
    say(f"big gemm T={T} E={E} k={k} N={N} K={K} {ty} gather={gather} drop={drop}")
    r = Routing(T, E, k, T + N, drop)
    g = torch.Generator(device=DEV).manual_seed(T + N + K)
    table = torch.from_numpy(oracle.e4m3_values()).to(DEV)
    small = torch.nonzero((table.abs() <= 8) & (table == table.round())).view(-1).to(torch.uint8)

    def codes(*shape):
        return small[torch.randint(0, len(small), shape, device=DEV, generator=g)]

    def scales(*shape):
        return 2.0 ** torch.randint(-1, 2, shape, device=DEV, generator=g).float()

    R, kb, nb = (T if gather else T * k), -(-K // 128), -(-N // 128)
    a = torch.full((R, K + 16), 127, dtype=torch.uint8, device=DEV)[:, :K]
    a.copy_(codes(R, K))
    w, sa, sw = codes(E, N, K), scales(R, kb), scales(E, nb, kb)
    outputs = []
    for _ in range(2):
        c = strided(T * k, N, TYPES[ty], 55.0, 3)
        apq.moe_fp8_gemm(a, sa, w, sw, c, expert_offsets=r.offsets if E > 1 else None,
                         sorted_pairs=r.pairs if gather else None, k=k)
        outputs.append(c)
    assert torch.equal(outputs[0], outputs[1])       # the same bits again
    assert bool((c[r.n:] == 55.0).all()) and bool((c.as_strided((T * k, 3), (N + 3, 1), N) == 55.0).all())
    source = (r.pairs[:r.n].long() // k) if gather else torch.arange(r.n, device=DEV)
    spread = torch.arange(K, device=DEV) // 128
    for e, rows in enumerate(r.groups):
        if len(rows) == 0:
            continue
        src = source[rows.start:rows.stop]
        ae = table[a[src].long()] * sa[src].double()[:, spread]
        we = table[w[e].long()] * sw[e].double().repeat_interleave(128, 0)[:N][:, spread]
        want = ae @ we.t().contiguous()
        assert torch.equal(c[rows.start:rows.stop], want.to(TYPES[ty]))


@pytest.mark.parametrize("T,E,N,K,ty", [(300, 64, 300, 272, "bf16"), (700, 512, 700, 400, "f32"), (5000, 16, 2600, 144, "f16")])
def test_gemm_when_one_expert_takes_all(T, E, N, K, ty):
    """Far more rows in one group than the average the launch goes by."""
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.full((T, 1), E - 2, dtype=torch.int32, device=DEV)
    ids[5], ids[T // 2] = 0, E - 1
    offsets, pairs = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
    apq.moe_group_by_expert(ids, E, offsets, pairs, torch.empty(E, dtype=torch.int32, device=DEV),
                            torch.empty(1, dtype=torch.int32, device=DEV))
    table = torch.from_numpy(oracle.e4m3_values()).to(DEV)
    small = torch.nonzero((table.abs() <= 8) & (table == table.round())).view(-1).to(torch.uint8)
    a = small[torch.randint(0, len(small), (T, K), device=DEV, generator=g)]
    w = small[torch.randint(0, len(small), (E, N, K), device=DEV, generator=g)]
    sa, sw = torch.ones(T, -(-K // 128), device=DEV), torch.ones(E, -(-N // 128), -(-K // 128), device=DEV)
    c = torch.empty(T, N, dtype=TYPES[ty], device=DEV)
    apq.moe_fp8_gemm(a, sa, w, sw, c, expert_offsets=offsets, sorted_pairs=pairs, k=1)
    order = pairs.long()
    for rows in (slice(0, 1), slice(1, T - 1), slice(T - 1, T)):
        e = int(ids[order[rows.start], 0])
        want = table[a[order[rows]].long()] @ table[w[e].long()].t().contiguous()
        assert torch.equal(c[rows], want.to(TYPES[ty]))


def test_gemm_gathers_without_groups():
    """sorted_pairs without expert_offsets: one group whose rows come from anywhere, some twice."""
    g = torch.Generator(device=DEV).manual_seed(2)
    for M, R, k, N, K in [(3, 2, 4, 40, 144), (50, 30, 2, 70, 256), (600, 90, 8, 8200, 272)]:
        pairs = torch.randint(0, R * k, (M,), dtype=torch.int32, device=DEV, generator=g)
        a = torch.randint(0, 80, (R, K), dtype=torch.uint8, device=DEV, generator=g)
        w = torch.randint(0, 80, (N, K), dtype=torch.uint8, device=DEV, generator=g)
        sa, sw = torch.ones(R, -(-K // 128), device=DEV), torch.ones(-(-N // 128), -(-K // 128), device=DEV)
        c = torch.empty(M, N, device=DEV)
        apq.moe_fp8_gemm(a, sa, w, sw, c, sorted_pairs=pairs, k=k)
        table = torch.from_numpy(oracle.e4m3_values()).to(DEV)
        want = (table[a.long()] @ table[w.long()].t().contiguous())[pairs.long() // k]
        size = (table[a.long()].abs() @ table[w.long()].abs().t().contiguous())[pairs.long() // k]
        assert bool(((c - want).abs() <= 2 * (K + 8) * U * size + U * want.abs()).all())


@pytest.mark.parametrize("ty", ["f16", "bf16", "f32"])
def test_rows_that_start_at_an_odd_element(ty):
    """Views one element into their memory: aligned to an element only."""
    T, E, k, H = 9, 4, 2, 150
    dt, r = TYPES[ty], Routing(T, E, k, 21, 0.1)
    g = torch.Generator(device=DEV).manual_seed(3)

    def odd(rows, cols, fill=None, dtype=dt):
        t = torch.full((rows * (cols + 2) + 1,), 5.0 if fill is None else fill, dtype=dtype, device=DEV)
        return t[1:].view(rows, cols + 2)[:, :cols]

    x, ys = odd(T, H), odd(T * k, H)
    x.copy_(torch.randn(T, H, device=DEV, generator=g))
    ys.copy_(torch.randn(T * k, H, device=DEV, generator=g))
    xs, rows = odd(T * k, H), torch.empty(T, k, dtype=torch.int32, device=DEV)
    apq.moe_permute_tokens(x, r.ids, r.offsets, r.pairs, xs, rows)
    assert torch.equal(xs[:r.n], x[dev(r.pairs_np // k).long()])
    got, want = odd(T, H), torch.empty(T, H, dtype=dt, device=DEV)
    apq.moe_unpermute_tokens(ys, rows, r.gates, got, add=x)
    apq.moe_unpermute_tokens(ys.contiguous(), rows, r.gates, want, add=x.contiguous())
    assert torch.equal(got, want)
    dys, dys2 = odd(T * k, H), torch.full((T * k, H), 5.0, dtype=dt, device=DEV)
    dg, dg2 = torch.empty(T, k, device=DEV), torch.empty(T, k, device=DEV)
    apq.moe_unpermute_tokens_backward(x, ys, rows, r.gates, dys, dg)
    apq.moe_unpermute_tokens_backward(x.contiguous(), ys.contiguous(), rows, r.gates, dys2, dg2)
    assert torch.equal(dys, dys2) and torch.equal(dg, dg2)
    q, q2 = odd(T, H, 0, torch.uint8), torch.empty(T, H, dtype=torch.uint8, device=DEV)
    s, s2 = torch.empty(T, 2, device=DEV), torch.empty(T, 2, device=DEV)
    apq.moe_fp8_quantize(x, q, s)
    apq.moe_fp8_quantize(x.contiguous(), q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    a, w = torch.zeros(T, 64, dtype=torch.uint8, device=DEV), torch.full((1, H, 64), 56, dtype=torch.uint8, device=DEV)
    a[:, 0] = 56                                      # 1.0
    c = odd(T, H)
    apq.moe_fp8_gemm(a, torch.ones(T, 1, device=DEV), w, torch.ones(1, 2, 1, device=DEV), c)
    assert bool((c == 1.0).all()) and bool((c.as_strided((T, 2), (H + 2, 1), c.storage_offset() + H) == 5.0).all())


def test_far_rows_of_a_large_array():
    """Sorted rows that lie more than 2^32 bytes (and 2^31 elements) into their array."""
    T, k, E, H = 40000, 8, 8, 8192                    # 320000 rows of 16 KiB: 5.2 GB
    ids = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k) % E
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    pairs = torch.empty(T * k, dtype=torch.int32, device=DEV)
    apq.moe_group_by_expert(ids, E, offsets, pairs, torch.empty(E, dtype=torch.int32, device=DEV),
                            torch.empty(1, dtype=torch.int32, device=DEV))
    x = (torch.arange(T, device=DEV)[:, None] % 251 + torch.arange(H, device=DEV) % 5).half()
    xs, rows = torch.empty(T * k, H, dtype=torch.float16, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    apq.moe_permute_tokens(x, ids, offsets, pairs, xs, rows)
    tail = slice(T * k - 500, T * k)
    assert torch.equal(xs[tail], x[pairs[tail].long() // k])
    dx = torch.empty_like(x)
    apq.moe_permute_tokens_backward(xs, rows, dx)
    assert torch.equal(dx, x * k)                     # sums up to 2040: exact in fp16
    dys, dg = torch.empty_like(xs), torch.empty(T, k, device=DEV)
    apq.moe_unpermute_tokens_backward(x, xs, rows, None, dys, dg)
    assert torch.equal(dys[tail], xs[tail])
    q, s = torch.empty(T * k, H, dtype=torch.uint8, device=DEV), torch.empty(T * k, H // 128, device=DEV)
    apq.moe_fp8_quantize(xs, q, s)
    q1, s1 = torch.empty(500, H, dtype=torch.uint8, device=DEV), torch.empty(500, H // 128, device=DEV)
    apq.moe_fp8_quantize(xs[tail], q1, s1)
    assert torch.equal(q[tail], q1) and torch.equal(s[tail], s1)
    # rows of a and c behind 2^31 bytes, read in place
    N = 8
    w, sw = torch.full((N, H), 56, dtype=torch.uint8, device=DEV), torch.ones(1, H // 128, device=DEV)
    c, c1 = torch.empty(T * k, N, device=DEV), torch.empty(500, N, device=DEV)
    apq.moe_fp8_gemm(q, s, w, sw, c)
    apq.moe_fp8_gemm(q1, s1, w, sw, c1)
    assert torch.equal(c[tail], c1)


@pytest.mark.parametrize("T", [2, 40, 700])
def test_gemm_nan_stays_in_its_row(T):
    """NaN in one row of a and one row of w reaches that row and that column of its expert only."""
    E, k, N, K = 3, 1, 150, 272
    r = Routing(T, E, k, 11 + T)
    a, sa, w, sw = _gemm_inputs(r, N, K, True, True, 5)
    victim = int(r.pairs_np[0])
    a[victim, 270] = 127
    e = next(e for e in range(E) if len(r.groups[e]))
    w[e, 149, 3] = 255
    c = f64(_gemm(r, a, sa, w, sw, "f32", True, N))
    clean_a, clean_w = a.copy(), w.copy()
    clean_a[victim, 270] = 0
    clean_w[e, 149, 3] = 0
    want, _, _ = oracle.fp8_gemm(clean_a, sa, clean_w, sw, r.groups, r.pairs_np)
    bad = np.zeros(want.shape, dtype=bool)
    bad[0] = True
    bad[r.groups[e].start:r.groups[e].stop, 149] = True
    assert np.isnan(c[bad]).all()
    np.testing.assert_array_equal(c[~bad], want[~bad])


def test_gemm_gradient_is_the_transposed_product():
    """dL/da = dc W through the same call with the weights and their scales transposed, against the
    float64 formula and against differences of the product itself (which is linear in a's scale)."""
    T, N, K = 48, 256, 384
    r = Routing(T, 2, 1, 8)
    a, sa, w, sw = _gemm_inputs(r, N, K, True, True, 9)
    rng = np.random.default_rng(10)
    table = oracle.e4m3_values()
    small = np.array([c for c in range(256) if abs(table[c]) <= 8 and table[c] == np.rint(table[c])], dtype=np.uint8)
    dc, sdc = rng.choice(small, size=(T, N)), np.ones((T, N // 128), dtype=np.float32)
    da = torch.empty(T, K, device=DEV)
    apq.moe_fp8_gemm(dev(dc), dev(sdc), dev(np.swapaxes(w, 1, 2).copy()), dev(np.swapaxes(sw, 1, 2).copy()), da,
                     expert_offsets=r.offsets)
    want = np.zeros((T, K))
    for e, rows in enumerate(r.groups):
        want[rows.start:rows.stop] = table[dc[rows.start:rows.stop]] @ oracle.fp8_dequantize(w[e], sw[e], 128)
    np.testing.assert_array_equal(f64(da), want)
    # the derivative along "row i's block b grows in proportion" is that block's part of <da, a>
    for i, b in [(0, 0), (20, 1), (47, 2)]:
        src = int(r.pairs_np[i])
        up, down = sa.copy(), sa.copy()
        up[src, b] *= 2
        down[src, b] *= 0
        d = (f64(_gemm(r, a, up, w, sw, "f32", True, N)) - f64(_gemm(r, a, down, w, sw, "f32", True, N)))[i] @ table[dc[i]] / 2
        cols = slice(b * 128, (b + 1) * 128)
        assert d == f64(da)[i, cols] @ (table[a[src, cols]] * sa[src, b])


# ------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------
class Ffn:
    """The experts' FFN on e4m3 weights: route, group, quantise, gate_up, silu, down, unpermute."""

    def __init__(self, T, E, k, H, I, seed):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        self.logits = dev(rng.standard_normal((T, E)).astype(np.float32))
        self.x = dev(rng.standard_normal((T, H)), torch.bfloat16)
        self.shared = dev(rng.standard_normal((T, H)), torch.bfloat16)

        def weights(n, kk):
            v = rng.standard_normal((E * n, kk)).astype(np.float32)
            m = np.abs(v).max()
            codes = oracle.e4m3_encode(v * (448 / m) * 0.999).reshape(E, n, kk)
            s = (np.exp(0.2 * rng.standard_normal((E, -(-n // 128), -(-kk // 128)))) * m / 448 / np.sqrt(kk)).astype(np.float32)
            return codes, s

        self.gu, self.gu_s = weights(2 * I, H)
        self.dn, self.dn_s = weights(H, I)
        self.dev_weights = [dev(t) for t in (self.gu, self.gu_s, self.dn, self.dn_s)]
        i32 = dict(dtype=torch.int32, device=DEV)
        P = T * k
        self.ids, self.gates = torch.empty(T, k, **i32), torch.empty(T, k, device=DEV)
        self.off, self.pairs = torch.empty(E + 1, **i32), torch.zeros(P, **i32)
        self.act, self.n = torch.empty(E, **i32), torch.empty(1, **i32)
        self.rows = torch.empty(T, k, **i32)
        self.xs = torch.empty(P, H, dtype=torch.bfloat16, device=DEV)
        self.q, self.qs = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(T, -(-H // 128), device=DEV)
        self.h = torch.empty(P, 2 * I, dtype=torch.bfloat16, device=DEV)
        self.aq, self.aqs = torch.empty(P, I, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(P, -(-I // 128), device=DEV)
        self.o = torch.empty(P, H, dtype=torch.bfloat16, device=DEV)
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)

    def run(self, stream=None):
        gu, gu_s, dn, dn_s = (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for t in self.dev_weights)
        kw = dict(stream=stream)
        apq.moe_route_topk(self.logits, self.k, self.ids, self.gates, **kw)
        apq.moe_group_by_expert(self.ids, self.E, self.off, self.pairs, self.act, self.n, **kw)
        apq.moe_permute_tokens(self.x, self.ids, self.off, self.pairs, self.xs, self.rows, **kw)
        apq.moe_fp8_quantize(self.x, self.q, self.qs, **kw)
        apq.moe_fp8_gemm(self.q, self.qs, gu, gu_s, self.h, expert_offsets=self.off, sorted_pairs=self.pairs, k=self.k, **kw)
        apq.moe_fp8_quantize_silu(self.h, self.aq, self.aqs, n_rows=self.off[self.E:], **kw)
        apq.moe_fp8_gemm(self.aq, self.aqs, dn, dn_s, self.o, expert_offsets=self.off, **kw)
        apq.moe_unpermute_tokens(self.o, self.rows, self.gates, self.y, add=self.shared, **kw)

    def outputs(self):
        return [t.clone() for t in (self.rows, self.xs, self.q, self.qs, self.h, self.aq, self.aqs, self.o, self.y)]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x,
                           y.view(torch.uint8) if y.element_size() == 1 else y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 384), (24, 16, 4, 384, 272), (200, 8, 2, 512, 256)])
def test_expert_ffn_run_step_by_step(T, E, k, H, I):
    """The whole run; every step against the oracle on that step's own inputs."""
    say(f"fp8 FFN T={T} E={E} k={k} H={H} I={I}")
    f = Ffn(T, E, k, H, I, 40 + T)
    f.run()
    ids, gates = oracle.route_topk(f.logits.cpu().numpy(), k)
    off, pairs, _, _ = oracle.group_by_expert(ids, E)
    rows = oracle.pair_rows(pairs, T * k, T * k).reshape(T, k)
    groups = [range(int(off[e]), int(off[e + 1])) for e in range(E)]
    np.testing.assert_array_equal(f.rows.cpu().numpy(), rows)
    assert torch.equal(f.xs, f.x[dev(np.asarray(pairs) // k).long()])
    codes, scales = oracle.fp8_quantize(f.x.float().cpu().numpy())
    np.testing.assert_array_equal(f.q.view(torch.uint8).cpu().numpy(), codes)
    np.testing.assert_array_equal(f.qs.cpu().numpy(), scales)

    def close(got, want, size, top, K):
        assert _worst(f64(got), want, size, top, K, "bf16") <= 1

    close(f.h, *oracle.fp8_gemm(codes, scales, f.gu, f.gu_s, groups, np.asarray(pairs) // k), H)
    h = f64(f.h)
    act = h[:, :I] / (1 + np.exp(-h[:, :I])) * h[:, I:]
    aq, aqs = f.aq.view(torch.uint8).cpu().numpy(), f.aqs.cpu().numpy()
    step = np.repeat(aqs.astype(np.float64), 128, axis=1)[:, :I]
    assert (np.abs(oracle.fp8_dequantize(aq, aqs) - act)
            <= np.maximum(2.0 ** -4 * np.abs(act), 2.0 ** -10 * step) * (1 + 32 * U) + 12 * U * np.abs(act)).all()
    close(f.o, *oracle.fp8_gemm(aq, aqs, f.dn, f.dn_s, groups, np.arange(T * k)), I)
    want, size = oracle.unpermute_tokens(f64(f.o), rows, f64(f.gates), f64(f.shared))
    assert (np.abs(f64(f.y) - want) <= HALF["bf16"] * np.abs(want) * (1 + 2 * k * U) + (k + 2) * U * size).all()


def test_expert_ffn_captured_replayed_and_on_another_stream():
    f = Ffn(24, 16, 4, 384, 272, 77)
    f.run()
    torch.cuda.synchronize()
    want = f.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (f.y, f.o, f.h, f.xs):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    f.run(stream=side)                      # the tensors belong to the current stream
    torch.cuda.current_stream().wait_stream(side)
    assert _same(f.outputs(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.run()
    logits, x = f.logits.clone(), f.x.clone()
    other = Ffn(24, 16, 4, 384, 272, 78)
    for turn in range(4):                   # replays on changed inputs, eager work in between
        f.logits.copy_(other.logits if turn % 2 else logits)
        f.x.copy_(other.x if turn % 2 else x)
        f.run()
        torch.cuda.synchronize()
        eager = f.outputs()
        for t in (f.y, f.o, f.h, f.xs):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(f.outputs(), eager)
        assert _same(f.outputs(), want) == (turn % 2 == 0)


def test_two_runs_at_once_on_two_streams():
    a, b = Ffn(16, 8, 2, 256, 256, 1), Ffn(40, 8, 2, 256, 256, 2)
    for f in (a, b):
        f.run()
    torch.cuda.synchronize()
    want = [a.outputs(), b.outputs()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for f, s in zip((a, b), streams):
            f.run(stream=s)
    torch.cuda.synchronize()
    assert _same(a.outputs(), want[0]) and _same(b.outputs(), want[1])


def test_large_runs_captured_and_at_once():
    """Sizes at which tokens are permuted by token and the products take whole tiles: captured and
    replayed on changed inputs, and two different runs at once on two streams."""
    a, b = Ffn(600, 8, 4, 512, 2048, 5), Ffn(900, 8, 4, 512, 2048, 6)
    want = []
    for f in (a, b):
        f.run()
        torch.cuda.synchronize()
        want.append(f.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for f in (a, b):
            for t in (f.y, f.o, f.h, f.xs):
                t.zero_()
        torch.cuda.synchronize()
        for f, s in zip((a, b), streams):
            f.run(stream=s)
        torch.cuda.synchronize()
        assert _same(a.outputs(), want[0]) and _same(b.outputs(), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    logits = a.logits.clone()
    for turn in range(3):
        a.logits.copy_(logits.flip(1) if turn % 2 else logits)
        a.run()
        torch.cuda.synchronize()
        eager = a.outputs()
        for t in (a.y, a.o, a.h, a.xs):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(a.outputs(), eager)
        assert _same(a.outputs(), want[0]) == (turn % 2 == 0)


def test_binding_refuses_shapes_and_types():
    T, E, k, H = 4, 8, 2, 64
    r = Routing(T, E, k, 1)
    x, xs, rows = torch.zeros(T, H, device=DEV), torch.zeros(T * k, H, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    q, s = torch.zeros(T, H, dtype=torch.uint8, device=DEV), torch.zeros(T, 1, device=DEV)
    w, ws = torch.zeros(E, 32, H, dtype=torch.uint8, device=DEV), torch.zeros(E, 1, 1, device=DEV)
    c = torch.zeros(T * k, 32, device=DEV)

    def refused(word, fn, *args, **kw):
        with pytest.raises(apq.MoeError, match=word) as err:
            fn(*args, **kw)
        assert err.value.code == apq.MOE_EINVAL

    refused("shape", apq.moe_permute_tokens, x, r.ids, r.offsets, r.pairs, xs[:-1], rows)
    refused("float16", apq.moe_permute_tokens, x, r.ids, r.offsets, r.pairs, xs.half(), rows)
    refused("int32", apq.moe_permute_tokens, x, r.ids.long(), r.offsets, r.pairs, xs, rows)
    refused("contiguous", apq.moe_permute_tokens, x.t().contiguous().t(), r.ids, r.offsets, r.pairs, xs, rows)
    refused("contiguous", apq.moe_permute_tokens, x, r.ids, r.offsets, r.pairs, xs, rows.t().contiguous().t())
    refused("not cuda", apq.moe_permute_tokens, x, r.ids.cpu(), r.offsets, r.pairs, xs, rows)
    refused("pair_rows has shape", apq.moe_permute_tokens_backward, xs, rows.view(-1), x)
    refused("gates", apq.moe_unpermute_tokens, xs, rows, r.gates.double(), x)
    refused("add", apq.moe_unpermute_tokens, xs, rows, None, x, add=x[:-1])
    refused("dgates", apq.moe_unpermute_tokens_backward, x, xs, rows, None, xs, r.gates[:-1])
    refused("NULL", apq.moe_unpermute_tokens_backward, x, xs, rows, None, None, None)
    refused("q is", apq.moe_fp8_quantize, x, q.int(), s)
    refused("scales", apq.moe_fp8_quantize, x, q, torch.zeros(T, 2, device=DEV))
    refused("n_rows", apq.moe_fp8_quantize, x, q, s, n_rows=r.offsets)
    refused("entries for 8 experts", apq.moe_fp8_gemm, q, s, w, ws, c, expert_offsets=r.offsets[:-1], sorted_pairs=r.pairs, k=k)
    refused("need expert_offsets", apq.moe_fp8_gemm, q, s, w, ws, c, sorted_pairs=r.pairs, k=k)
    refused("a has 4 rows", apq.moe_fp8_gemm, q, s, w, ws, c, expert_offsets=r.offsets)
    refused("w needs", apq.moe_fp8_gemm, q, s, w[:, :, ::2], ws, c, expert_offsets=r.offsets, sorted_pairs=r.pairs, k=k)
    refused("w_scales", apq.moe_fp8_gemm, q, s, w, ws[:-1], c, expert_offsets=r.offsets, sorted_pairs=r.pairs, k=k)


def test_empty_calls():
    e32, i32 = torch.zeros(0, 64, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    off = torch.zeros(9, dtype=torch.int32, device=DEV)
    apq.moe_permute_tokens(e32, i32, off, i32.view(-1), e32, i32)
    apq.moe_permute_tokens_backward(e32, i32, e32)
    apq.moe_unpermute_tokens(e32, i32, None, e32)
    apq.moe_unpermute_tokens_backward(e32, e32, i32, None, e32, torch.zeros(0, 2, device=DEV))
    q, s = torch.zeros(0, 64, dtype=torch.uint8, device=DEV), torch.zeros(0, 1, device=DEV)
    apq.moe_fp8_quantize(e32, q, s)
    w, ws = torch.zeros(8, 32, 64, dtype=torch.uint8, device=DEV), torch.zeros(8, 1, 1, device=DEV)
    apq.moe_fp8_gemm(q, s, w, ws, torch.zeros(0, 32, device=DEV), expert_offsets=off)
    torch.cuda.synchronize()
