"""The 8-bit linear layer (include/fp8.h) against plain implementations in 64 bits.

Tolerances, per value:
  * E4M3 codes: half a step is 2^-4 of the value, or half of the smallest step
    2^-9 times the block's scale; BF16 outputs: 2^-8 of the value.
  * the norm's v: its fp32 sum of squares adds at most 32 + 13 terms in a chain
    (long rows: 8 per 8192 columns), so v is off by at most 2^-18 of itself.
  * silu: __expf is off by 2 + 1.173 |x| ulp (111 ulp at |x| = 90, 2^-16), the
    fast division by 2 ulp: 2^-15 together.
  * the products: exact products, summed per 128 on the tensor cores and over
    blocks in fp32; 2^-10 of sum |x w| (the tolerance of the library's other
    GEMMs) and the rounding to BF16.  Products of small whole numbers add up
    without any rounding, so there the outputs have to be equal.
"""
import pytest
import torch

from gpu_util import guarded_empty

pytestmark = pytest.mark.gpu
F8, BF16, F32, F64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def nv():
    import gemm_decode_nvfp4_b200 as m
    assert torch.cuda.is_available()
    yield m
    m.check_device_errors()


def randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(BF16).cuda()


def blocks(n):
    return (n + 127) // 128


def e4m3(v):
    """fp64 -> nearest E4M3 value (ties to even, saturating)."""
    v = v.clamp(-448.0, 448.0)
    step = torch.exp2(torch.clamp(torch.frexp(v)[1].double() - 4, min=-9))
    return torch.round(v / step) * step


def per_block(v, rows):
    """max |v| per `rows` rows and 128 columns."""
    R, K = v.shape
    a = torch.zeros((blocks(R) * 128 if rows == 128 else R, blocks(K) * 128), dtype=v.dtype, device=v.device)
    a[:R, :K] = v.abs()
    return a.view(-1, rows, blocks(K), 128).amax((1, 3))


def spread(s, rows, R, K):
    return s.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :K]


def check_rule(w, q, s, rows):
    """q, s bit for bit the rule's, of exactly known values w."""
    R, K = w.shape
    a = per_block(w.float(), rows)
    # (divided by a tensor: torch divides by a number on the GPU by multiplying with its reciprocal)
    s_ref = torch.clamp(a / torch.full_like(a, 448.0), min=2.0 ** -126)
    assert torch.equal(s, s_ref)
    v = w.float() * spread(torch.ones_like(s_ref) / s_ref, rows, R, K)   # fp32, as the rule says
    assert torch.equal(q.double(), e4m3(v.double()))


def check_quantized(v, q, s, rel):
    """q * s within half an E4M3 step of the fp64 v, which the kernel knows to `rel`."""
    K = v.shape[1]
    s_ref = torch.clamp(per_block(v, 1) / 448.0, min=2.0 ** -126)
    assert bool(((s.double() - s_ref).abs() <= s_ref * (rel + 2.0 ** -23)).all())
    sv = spread(s.double(), 1, v.shape[0], K)
    tol = v.abs() * (2.0 ** -4 + 2 * rel + 2.0 ** -22) + sv * 2.0 ** -10
    bad = (q.double() * sv - v).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} codes out of tolerance"


# ---------------------------------------------------------------- quantizers

@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (17, 2064), (300, 5120), (1, 17408), (2049, 400)])
def test_quantize_is_the_rule(nv, M, K):
    x = randn((M, K), M + K)
    q, chk_q = guarded_empty((M, K), F8)
    s, chk_s = guarded_empty((M, blocks(K)), F32)
    nv.fp8_quantize(x, q, s)
    check_rule(x, q, s, 1)
    chk_q(), chk_s()


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (127, 272), (1001, 2064), (384, 1024)])
def test_quantize_weights_is_the_rule(nv, N, K):
    w = randn((N, K), N + K, 0.02)
    q, chk_q = guarded_empty((N, K), F8)
    s, chk_s = guarded_empty((blocks(N), blocks(K)), F32)
    nv.fp8_quantize_weights(w, q, s)
    check_rule(w, q, s, 128)
    chk_q(), chk_s()


@pytest.mark.parametrize("M,K", [(1, 16), (5, 144), (64, 2064), (8, 17408), (700, 1024)])
def test_gated_quantize(nv, M, K):
    x = randn((M, 2 * K), M + K, 2.0)
    q, s = nv.fp8_quantize_new(x, gated=True)
    g, u = x[:, :K].double(), x[:, K:].double()
    check_quantized(g * torch.sigmoid(g) * u, q, s, 2.0 ** -15)


def test_gated_quantize_far_gates(nv):
    """Gates from -120 to 120: exp overflows below -88, where silu is zero."""
    g = torch.linspace(-120, 120, 512).to(BF16)
    x = torch.cat([g.repeat(3, 1), torch.ones(3, 512, dtype=BF16)], 1).cuda()
    q, s = nv.fp8_quantize_new(x, gated=True)
    gd = g.double().cuda().repeat(3, 1)
    check_quantized(gd * torch.sigmoid(gd), q, s, 2.0 ** -15)


@pytest.mark.parametrize("gated", [False, True])
def test_quantize_rows_of_a_wider_tensor(nv, gated):
    K = 272
    wide = randn((33, 1024), 5)
    x = wide[:, 64:64 + K * (2 if gated else 1)]
    q, s = nv.fp8_quantize_new(x, gated=gated)
    q2, s2 = nv.fp8_quantize_new(x.contiguous(), gated=gated)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    w = wide[:, 8:8 + K]
    a, b = nv.fp8_quantize_weights_new(w), nv.fp8_quantize_weights_new(w.contiguous())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_quantize_zero_tiny_and_large_blocks(nv):
    """An all-zero block, subnormal BF16 values and values near BF16's maximum."""
    x = torch.zeros((4, 512), dtype=BF16)
    x[0, 128:256] = 2.0 ** -133
    x[1, :128] = (3.3e38 * torch.linspace(-1, 1, 128, dtype=F64)).to(BF16)
    x[2, 300] = -1.0
    x = x.cuda()
    q, s = nv.fp8_quantize_new(x)
    check_rule(x, q, s, 1)
    qw, sw = nv.fp8_quantize_weights_new(x)
    check_rule(x, qw, sw, 128)


def test_quantize_nan_and_infinity(nv):
    """NaN stays in its own element; an infinity takes its own block only."""
    x = randn((2, 384), 3)
    x[0, 5] = float("nan")
    x[1, 200] = float("inf")
    clean = x.clone()
    clean[0, 5], clean[1, 200] = 0.0, 0.0
    q, s = nv.fp8_quantize_new(x)
    q0, s0 = nv.fp8_quantize_new(clean)
    same = torch.ones_like(q, dtype=torch.bool)
    same[0, 5] = False
    same[1, 128:256] = False
    assert torch.equal(q.float()[same], q0.float()[same])
    assert bool(q.float()[0, 5].isnan()) and bool(q.float()[1, 200].isnan())
    assert s[1, 1].item() == float("inf")
    s[1, 1] = s0[1, 1]
    assert torch.equal(s, s0)


# ----------------------------------------------------------------------- norm

def norm_ref(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).to(BF16)
    hd = h.double()
    return h, hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps) * w.double()


def check_y(v, y):
    assert bool(((y.double() - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -133).all())


@pytest.mark.parametrize("M,K", [(1, 16), (5, 128), (3, 256), (9, 272), (4, 512), (6, 1024), (5, 1040), (2, 5120),
                                 (3, 8192), (2, 8208), (2, 16384), (3, 17408), (1, 32768), (2, 32784), (1, 65552)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(nv, M, K, residual):
    x, w = randn((M, K), M + K), randn((K,), K)
    r = randn((M, K), M + K + 1, 3.0) if residual else None
    h, v = norm_ref(x, r, w, 1e-6)
    q, chk_q = guarded_empty((M, K), F8)
    s, chk_s = guarded_empty((M, blocks(K)), F32)
    y, chk_y = guarded_empty((M, K), BF16)
    ro, chk_r = guarded_empty((M, K), BF16)
    nv.fp8_rmsnorm(x, w, 1e-6, residual=r, residual_out=ro if residual else None, y=y, q=q, s=s)
    check_y(v, y)
    check_quantized(v, q, s, 2.0 ** -18)
    if residual:
        assert torch.equal(ro, h)
    chk_q(), chk_s(), chk_y(), chk_r()


@pytest.mark.parametrize("M,K", [(297, 1040), (700, 5120), (600, 8192), (900, 8208), (1200, 16384), (305, 17408),
                                 (301, 32768), (2500, 272)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_many_rows(nv, M, K, residual):
    """More rows than CTAs: each CTA takes several, out of strided tensors."""
    wide = randn((M, K + 24), M + K)
    x, w = wide[:, 8:8 + K], randn((K,), K)
    r = randn((M, K + 8), M + K + 1, 3.0)[:, :K] if residual else None
    h, v = norm_ref(x, r, w, 1e-6)
    q, chk_q = guarded_empty((M, K), F8)
    s, chk_s = guarded_empty((M, blocks(K)), F32)
    y, chk_y = guarded_empty((M, K), BF16)
    ro, chk_r = guarded_empty((M, K), BF16)
    nv.fp8_rmsnorm(x, w, 1e-6, residual=r, residual_out=ro if residual else None, y=y, q=q, s=s)
    check_y(v, y)
    check_quantized(v, q, s, 2.0 ** -18)
    if residual:
        assert torch.equal(ro, h)
        nv.fp8_rmsnorm(x, w, 1e-6, residual=r, y=y)      # in place
        assert torch.equal(r, h)
    chk_q(), chk_s(), chk_y(), chk_r()


@pytest.mark.parametrize("K", [400, 5120, 40960])
def test_rmsnorm_outputs_alone_and_in_place(nv, K):
    """y alone, (q, s) alone and the residual in place give what all together give."""
    M = 7
    x, w, r = randn((M, K), 1), randn((K,), 2), randn((M, K), 3)
    new = lambda: (torch.empty((M, K), dtype=F8, device="cuda"),  # noqa: E731
                   torch.empty((M, blocks(K)), dtype=F32, device="cuda"))
    q, s = new()
    y, ro = torch.empty_like(x), torch.empty_like(x)
    nv.fp8_rmsnorm(x, w, 1e-5, residual=r, residual_out=ro, y=y, q=q, s=s)
    y2, r2 = torch.empty_like(x), r.clone()
    nv.fp8_rmsnorm(x, w, 1e-5, residual=r2, y=y2)
    assert torch.equal(y, y2) and torch.equal(r2, ro)
    (q3, s3), r3 = new(), r.clone()
    nv.fp8_rmsnorm(x, w, 1e-5, residual=r3, q=q3, s=s3)
    assert torch.equal(q.view(torch.uint8), q3.view(torch.uint8)) and torch.equal(s, s3) and torch.equal(r3, ro)


def test_rmsnorm_strides(nv):
    wide = randn((20, 4096), 9)
    x, r = wide[:, :528], wide[:, 1024:1552]
    out = torch.zeros((20, 4096), dtype=BF16, device="cuda")
    y, ro = out[:, 8:536], out.clone()[:, 2048:2576]
    w = randn((528,), 4)
    nv.fp8_rmsnorm(x, w, 1e-6, residual=r, residual_out=ro, y=y)
    h, v = norm_ref(x, r, w, 1e-6)
    assert torch.equal(ro, h)
    check_y(v, y)
    assert not bool(out[:, :8].any()) and not bool(out[:, 536:].any())


def test_rmsnorm_zero_row_and_nan_row(nv):
    """A zero row gives zeros (eps = 0: 0 / 0 = NaN, as the formula says); a NaN stays in its row."""
    x = randn((3, 640), 6)
    x[0] = 0.0
    x[1, 17] = float("nan")
    w = randn((640,), 7)
    y = torch.empty_like(x)
    nv.fp8_rmsnorm(x, w, 1e-6, y=y)
    assert not bool(y[0].any()) and bool(y[1].isnan().all())
    check_y(norm_ref(x[2:], None, w, 1e-6)[1], y[2:])
    nv.fp8_rmsnorm(x, w, 0.0, y=y)
    assert bool(y[0].isnan().all())


# ------------------------------------------------------------------- products

def values(q, s, rows):
    return q.double() * spread(s.double(), rows, *q.shape)


def check_product(y, x, w, what=""):
    """y against x . w^T in 64 bits, x and w the dequantized values."""
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    bad = (y.double() - ref).abs() > mag * 2.0 ** -10 + ref.abs() * 2.0 ** -8
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outputs out of tolerance, first at " \
                                f"{[int(i) for i in bad.nonzero()[0]]}"


def whole_numbers(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g).float().to(F8).cuda()


def powers(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.randint(-1, 2, shape, generator=g).float()).cuda()


SHAPES = [(1, 128, 128), (1, 1, 16), (2, 130, 144), (16, 256, 512), (17, 1001, 2064), (32, 384, 1040),
          (33, 129, 5120), (64, 5120, 640), (65, 257, 400), (128, 128, 4096), (129, 512, 1024), (200, 5120, 1024),
          (300, 17408, 256), (1000, 8192, 400), (1025, 4099, 1040), (4100, 640, 272), (1, 17408, 5120),
          (47, 5120, 17408), (3, 640, 65552)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_whole_numbers_are_exact(nv, M, N, K):
    """Sums of products of small whole numbers with power-of-two scales are exact
    in fp32, whatever the order: the output is their BF16 rounding."""
    x, w = whole_numbers((M, K), M + K), whole_numbers((N, K), N + K)
    sx, sw = powers((M, blocks(K)), M), powers((blocks(N), blocks(K)), N)
    Y, chk = guarded_empty((M, N), BF16)
    for static in (False, True):
        Y.fill_(float("nan"))
        nv.fp8_gemm(x, sx, w, sw, Y, static_weights=static)
        ref = (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16)
        assert torch.equal(Y, ref), f"{int((Y != ref).sum())} of {ref.numel()} differ"
    chk()


@pytest.mark.parametrize("M,N,K", [(200, 130, 2064), (90, 1001, 2064), (90, 2560, 5120), (90, 5125, 5120),
                                   (128, 1001, 5120), (64, 5125, 2064), (90, 17408, 528), (130, 5125, 5120),
                                   (128, 5125, 2064), (130, 2560, 5120), (384, 1001, 5120), (128, 17411, 2064),
                                   (256, 5120, 2064), (100, 5125, 17408), (250, 5120, 17408)])
def test_gemm_every_tile_width_and_split(nv, M, N, K):
    """Middle sizes, where every tile width and split of k is chosen for some."""
    x, w = whole_numbers((M, K), M + K), whole_numbers((N, K), N + K)
    sx, sw = powers((M, blocks(K)), M), powers((blocks(N), blocks(K)), N)
    Y, chk = guarded_empty((M, N), BF16)
    nv.fp8_gemm(x, sx, w, sw, Y)
    assert torch.equal(Y, (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16))
    chk()


@pytest.mark.parametrize("T,E,N,K", [(1000, 8, 1536, 1040), (900, 4, 1540, 1040), (2000, 20, 1536, 144),
                                     (900, 4, 1536, 4112), (2000, 20, 1001, 144), (700, 5, 1001, 1040)])
def test_grouped_every_tile_width(nv, T, E, N, K):
    g = torch.Generator().manual_seed(T + E)
    ends = [0, *sorted(torch.randint(0, T + 1, (E - 1,), generator=g).tolist()), T - 3]
    ends = [min(e, T - 3) for e in ends]
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, blocks(K)), 3), powers((E, blocks(N), blocks(K)), 4)
    Y, chk = guarded_empty((T, N), BF16)
    Y.fill_(5.0)
    ref = grouped_ref(x, sx, w, sw, ends, Y)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    assert torch.equal(Y, ref)
    chk()


@pytest.mark.parametrize("M,N,K", [(1, 1001, 5120), (20, 5120, 2064), (60, 300, 17408), (100, 700, 4096),
                                   (520, 17408, 1040), (1111, 4097, 2048)])
def test_gemm_random(nv, M, N, K):
    X, W = randn((M, K), M), randn((N, K), N, 0.02)
    w, sw = nv.fp8_quantize_weights_new(W)
    q, s = nv.fp8_quantize_new(X)
    Y = nv.fp8_linear(X, w, sw)
    check_product(Y, values(q, s, 1), values(w, sw, 128))
    Y2 = torch.empty_like(Y)
    nv.fp8_gemm(q, s, w, sw, Y2)
    assert torch.equal(Y, Y2)          # deterministic, split or not
    assert torch.equal(nv.fp8_linear(X[0], w, sw), nv.fp8_linear(X[:1], w, sw)[0])


@pytest.mark.parametrize("M,N", [(5, 700), (40, 129), (1500, 5125)])
def test_gemm_wider_output(nv, M, N):
    """Y inside a wider tensor at an odd column: nothing beside it is written."""
    K = 400
    x, w = whole_numbers((M, K), 1), whole_numbers((N, K), 2)
    sx, sw = powers((M, 4), 3), powers((blocks(N), 4), 4)
    wide = torch.full((M, N + 9), 7.0, dtype=BF16, device="cuda")
    nv.fp8_gemm(x, sx, w, sw, wide[:, 3:3 + N])
    assert torch.equal(wide[:, 3:3 + N], (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16))
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + N:] == 7).all())


@pytest.mark.parametrize("M,N", [(4, 300), (100, 300), (1500, 5000)])
def test_gemm_nan_stays_in_its_row_and_column(nv, M, N):
    K = 528
    x, w = whole_numbers((M, K), 1), whole_numbers((N, K), 2)
    sx, sw = powers((M, 5), 3), powers((blocks(N), 5), 4)
    ref = (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16)
    x.view(torch.uint8)[1, 527] = 0x7F
    w.view(torch.uint8)[N - 1, 3] = 0xFF
    Y = torch.empty((M, N), dtype=BF16, device="cuda")
    nv.fp8_gemm(x, sx, w, sw, Y)
    assert bool(Y[1].isnan().all()) and bool(Y[:, N - 1].isnan().all())
    Y[1], ref[1] = 0, 0
    Y[:, N - 1], ref[:, N - 1] = 0, 0
    assert torch.equal(Y, ref)


def grouped_ref(x, sx, w, sw, ends, Y):
    ref, X = Y.clone(), values(x, sx, 1)
    for e in range(w.shape[0]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            ref[a:b] = (X[a:b] @ values(w[e], sw[e], 128).T).float().to(BF16)
    return ref


COUNTS = [
    ([1], 1), ([0, 0, 3, 0], 3), ([0, 0], 5), ([17, 0, 1, 128, 129, 5, 0], 300), ([3] * 40, 130), ([64] * 8, 512),
    ([700, 0, 1, 300], 1024), ([2100, 5, 0, 1999], 4104), ([1] * 200, 200), ([150] * 20, 3001),
]


@pytest.mark.parametrize("counts,T", COUNTS)
@pytest.mark.parametrize("N,K", [(128, 128), (300, 144), (1001, 1040)])
@pytest.mark.parametrize("start", [0, 2])
def test_grouped_whole_numbers_are_exact(nv, counts, T, N, K, start):
    """Every row is its expert's product; rows before the first and behind the
    last expert's keep what they hold."""
    E = len(counts)
    ends = [start]
    for c in counts:
        ends.append(ends[-1] + c)
    T = max(T, ends[-1])
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, blocks(K)), 3), powers((E, blocks(N), blocks(K)), 4)
    Y, chk = guarded_empty((T, N), BF16)
    Y.fill_(5.0)
    ref = grouped_ref(x, sx, w, sw, ends, Y)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    assert torch.equal(Y, ref), f"{int((Y != ref).any(1).sum())} rows differ"
    chk()


def test_grouped_nan_rows_elsewhere(nv):
    """NaN in another expert's weights and in rows of no expert reach nothing."""
    E, N, K, T = 3, 200, 272, 50
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, 3), 3), powers((E, 2, 3), 4)
    w.view(torch.uint8)[1], sw[1] = 0x7F, float("nan")
    x.view(torch.uint8)[40:], sx[40:] = 0x7F, float("nan")
    Y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    ends = [0, 20, 20, 40]
    ref = grouped_ref(x, sx, w, sw, ends, Y)
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    assert torch.equal(Y, ref) and not bool(Y.isnan().any())


@pytest.mark.parametrize("ends", [[0, 30, 10, 40], [-5, 10, 20, 40], [0, 10, 20, 1000], [50, 0, 50, 0],
                                  [-(1 << 31), (1 << 31) - 1, 0, 7]])
def test_grouped_bad_offsets_are_clamped_and_counted(nv, ends):
    """Offsets that decrease or leave the rows: counted, and nothing outside Y is touched."""
    E, N, K, T = 3, 136, 144, 50
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, 2), 3), powers((E, 2, 2), 4)
    Y, chk = guarded_empty((T, N), BF16)
    nv.check_device_errors()
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    torch.cuda.synchronize()
    with pytest.raises(nv.Nvfp4Error, match="offsets"):
        nv.check_device_errors()
    chk()
    nv.check_device_errors()   # read once


@pytest.mark.parametrize("E", [1, 33, 1000, 4096])
def test_grouped_many_experts(nv, E):
    """One row for every third expert, up to the largest number of experts."""
    N, K = 16, 32
    ends = [0]
    for e in range(E):
        ends.append(ends[-1] + (e % 3 == 0))
    T = ends[-1]
    x, w = whole_numbers((T, K), 1), whole_numbers((E, N, K), 2)
    sx, sw = powers((T, 1), 3), powers((E, 1, 1), 4)
    Y = torch.zeros((T, N), dtype=BF16, device="cuda")
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    e = torch.arange(0, E, 3, device="cuda")
    ref = torch.einsum("tk,tnk->tn", x.double() * sx.double(), w[e].double() * sw[e].double())
    assert torch.equal(Y, ref.float().to(BF16))


def test_grouped_equals_dense(nv):
    """An expert's rows give what the dense product of those rows gives, within the tolerance."""
    E, N, K, T = 4, 768, 1024, 600
    X, W = randn((T, K), 1), randn((E * N, K), 2, 0.02)
    x, sx = nv.fp8_quantize_new(X)
    w, sw = nv.fp8_quantize_weights_new(W)
    w, sw = w.view(E, N, K), sw.view(E, N // 128, K // 128)
    ends = [0, 13, 13, 400, 600]
    Y = torch.empty((T, N), dtype=BF16, device="cuda")
    nv.fp8_gemm_grouped(x, sx, w, sw, torch.tensor(ends, dtype=torch.int32, device="cuda"), Y)
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if b > a:
            check_product(Y[a:b], values(x[a:b], sx[a:b], 1), values(w[e], sw[e], 128), f"expert {e}")


@pytest.mark.parametrize("M,N,K", [(5, 300, 1024), (100, 700, 512), (900, 4100, 2048), (900, 4100, 2064)])
def test_scales_at_any_4_byte_address(nv, M, N, K):
    """Scales that start at odd multiples of 4 bytes, dense and grouped."""
    x, w = whole_numbers((M, K), 1), whole_numbers((N, K), 2)
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    sx, sw = powers((M, blocks(K)), 3), powers((blocks(N), blocks(K)), 4)
    ref = (values(x, sx, 1) @ values(w, sw, 128).T).float().to(BF16)
    ends = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    for a, b in ((off(sx), sw), (sx, off(sw)), (off(sx), off(sw))):
        Y = torch.empty((M, N), dtype=BF16, device="cuda")
        nv.fp8_gemm(x, a, w, b, Y)
        assert torch.equal(Y, ref)
        Y.fill_(0)
        nv.fp8_gemm_grouped(x, a, w[None], b[None], ends, Y)
        assert torch.equal(Y, ref)


def test_elements_past_32_bits(nv):
    """Tensors of more than 2^32 elements: the last rows are what a small call gives."""
    M, K, n = 270000, 16384, 3
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    x[-n:] = randn((n, K), 1)
    w = randn((K,), 2)
    q, s = torch.empty((M, K), dtype=F8, device="cuda"), torch.empty((M, K // 128), dtype=F32, device="cuda")
    nv.fp8_quantize(x, q, s)
    q1, s1 = nv.fp8_quantize_new(x[-n:])
    assert torch.equal(q[-n:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-n:], s1)
    nv.fp8_rmsnorm(x, w, q=q, s=s)
    nv.fp8_rmsnorm(x[-n:], w, q=q1, s=s1)
    assert torch.equal(q[-n:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-n:], s1)
    nv.fp8_quantize_weights(x, q, s[:blocks(M)])
    q2, s2 = nv.fp8_quantize_weights_new(x[M // 128 * 128:])
    assert torch.equal(q[M // 128 * 128:].view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s[blocks(M) - 1:blocks(M)], s2)
    del x
    # as activations, as weights of the last expert, and with a far row of Y
    wq, sw = whole_numbers((130, K), 3), powers((2, K // 128), 4)
    Y = torch.empty((M, 130), dtype=BF16, device="cuda")
    nv.fp8_gemm(q, s, wq, sw, Y)
    Y1 = torch.empty((M % 128, 130), dtype=BF16, device="cuda")
    nv.fp8_gemm(q[M // 128 * 128:], s[M // 128 * 128:], wq, sw, Y1)
    check_product(Y[M // 128 * 128:], values(q[M // 128 * 128:], s[M // 128 * 128:], 1), values(wq, sw, 128))
    E, N = 100, 2700
    xs, ss = whole_numbers((5, K), 5), powers((5, K // 128), 6)
    we, se = q.view(E, N, K), powers((E, blocks(N), K // 128), 7)
    we[E - 1] = whole_numbers((N, K), 8)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 5
    wide = torch.zeros((5, 1 << 30), dtype=BF16, device="cuda")
    nv.fp8_gemm_grouped(xs, ss, we, se, offsets, wide[:, :N])
    ref = (values(xs, ss, 1) @ values(we[E - 1], se[E - 1], 128).T).float().to(BF16)
    assert torch.equal(wide[:, :N], ref)


# ------------------------------------------------------------- empty, together

def test_empty_calls(nv):
    e = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    nv.fp8_quantize(e(0, 128, dtype=BF16), e(0, 128, dtype=F8), e(0, 1, dtype=F32))
    nv.fp8_quantize_weights(e(0, 128, dtype=BF16), e(0, 128, dtype=F8), e(0, 1, dtype=F32))
    nv.fp8_rmsnorm(e(0, 128, dtype=BF16), e(128, dtype=BF16), y=e(0, 128, dtype=BF16))
    w, sw = whole_numbers((64, 128), 1), powers((1, 1), 1)
    nv.fp8_gemm(e(0, 128, dtype=F8), e(0, 1, dtype=F32), w, sw, e(0, 64, dtype=BF16))
    nv.fp8_gemm_grouped(e(0, 128, dtype=F8), e(0, 1, dtype=F32), w[None], sw[None],
                        torch.zeros(2, dtype=torch.int32, device="cuda"), e(0, 64, dtype=BF16))
    torch.cuda.synchronize()


def test_refusals_on_the_device(nv):
    x, w = whole_numbers((4, 128), 1), whole_numbers((64, 128), 2)
    sx, sw = powers((4, 1), 1), powers((1, 1), 2)
    Y = torch.empty((4, 64), dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        nv.fp8_gemm(x, sx, w[:, :64], sw, Y)
    with pytest.raises(ValueError):
        nv.fp8_gemm(x, sx[:2], w, sw, Y)
    with pytest.raises(ValueError):
        nv.fp8_gemm(x, sx, w, sw, Y[:, :32])
    with pytest.raises(TypeError):
        nv.fp8_gemm(x.view(torch.uint8), sx, w, sw, Y)
    with pytest.raises(ValueError):
        nv.fp8_gemm_grouped(x, sx, w[None], sw[None], torch.zeros(3, dtype=torch.int32, device="cuda"), Y)
    X = randn((4, 128), 1)
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_rmsnorm(X, X[0], y=X)                       # y over x
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_rmsnorm(X, X[0].clone())                    # no output
    with pytest.raises(nv.Nvfp4Error):
        nv.fp8_rmsnorm(X[:1].expand(4, 128), X[0].clone(), y=torch.empty_like(X))   # rows on top of each other
    with pytest.raises(ValueError):
        nv.fp8_rmsnorm(X, X[0].clone(), q=x)
    with pytest.raises(ValueError):
        nv.fp8_rmsnorm(X, X[0].clone(), residual_out=torch.empty_like(X), y=torch.empty_like(X))


def mlp(nv, st):
    """One gated MLP of a decoder layer: norm, up product, gated quantize, down product."""
    nv.fp8_rmsnorm(st["x"], st["nw"], 1e-6, residual=st["r"], residual_out=st["h"], q=st["q"], s=st["s"])
    nv.fp8_gemm(st["q"], st["s"], st["wu"], st["su"], st["gu"], static_weights=True)
    nv.fp8_quantize(st["gu"], st["q2"], st["s2"], gated=True)
    nv.fp8_gemm(st["q2"], st["s2"], st["wd"], st["sd"], st["y"], static_weights=True)


def mlp_state(nv, M, H, I, seed):
    new = lambda dtype, *shape: torch.full(shape, 0, dtype=dtype, device="cuda")  # noqa: E731
    st = {"x": randn((M, H), seed), "r": randn((M, H), seed + 1), "nw": randn((H,), seed + 2)}
    st["wu"], st["su"] = nv.fp8_quantize_weights_new(randn((2 * I, H), 11, 0.02))
    st["wd"], st["sd"] = nv.fp8_quantize_weights_new(randn((H, I), 12, 0.02))
    st |= {"h": new(BF16, M, H), "q": new(F8, M, H), "s": new(F32, M, blocks(H)), "gu": new(BF16, M, 2 * I),
           "q2": new(F8, M, I), "s2": new(F32, M, blocks(I)), "y": new(BF16, M, H)}
    return st


def check_mlp(st):
    """Each step against its definition, on what the step before left."""
    h, v = norm_ref(st["x"], st["r"], st["nw"], 1e-6)
    assert torch.equal(st["h"], h)
    check_quantized(v, st["q"], st["s"], 2.0 ** -18)
    check_product(st["gu"], values(st["q"], st["s"], 1), values(st["wu"], st["su"], 128), "up")
    I = st["q2"].shape[1]
    g, u = st["gu"][:, :I].double(), st["gu"][:, I:].double()
    check_quantized(g * torch.sigmoid(g) * u, st["q2"], st["s2"], 2.0 ** -15)
    check_product(st["y"], values(st["q2"], st["s2"], 1), values(st["wd"], st["sd"], 128), "down")


@pytest.mark.parametrize("M", [1, 37, 700])
def test_mlp_as_used(nv, M):
    st = mlp_state(nv, M, 1024, 1808, 20)
    mlp(nv, st)
    check_mlp(st)


@pytest.mark.parametrize("M", [1, 300])
def test_mlp_captured_and_replayed(nv, M):
    """A captured graph replayed on new inputs, also while another graph of the
    same shapes runs on a second stream."""
    sts = [mlp_state(nv, M, 1024, 1808, 30 + i) for i in range(2)]
    for st in sts:
        mlp(nv, st)
    torch.cuda.synchronize()
    graphs = []
    for st in sts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mlp(nv, st)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sts]
    for rep in range(3):
        for i, st in enumerate(sts):
            st["x"].copy_(randn((M, 1024), 100 + 10 * rep + i))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for st in sts:
            check_mlp(st)


def test_calls_on_a_side_stream_are_ordered(nv):
    """Each call waits for what its own stream wrote before it, many times over."""
    st = mlp_state(nv, 5, 1024, 528, 50)
    s = torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        xs = [randn((5, 1024), 60 + i) for i in range(20)]
        for x in xs:
            st["x"].copy_(x)
            mlp(nv, st)
            outs.append(st["y"].clone())
    s.synchronize()
    for x, y in zip(xs, outs):
        st["x"].copy_(x)
        mlp(nv, st)
        torch.cuda.synchronize()
        assert torch.equal(st["y"], y)


def test_moe_as_used(nv):
    """Tokens sorted by expert: up product, gated quantize and down product per expert."""
    E, H, I, tokens, top = 8, 512, 400, 70, 2
    X = randn((tokens, H), 70)
    g = torch.Generator().manual_seed(1)
    experts = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(tokens)]).cuda()
    order = experts.flatten().argsort(stable=True)
    counts = torch.bincount(experts.flatten(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    up = [nv.fp8_quantize_weights_new(randn((2 * I, H), 80 + e, 0.05)) for e in range(E)]
    down = [nv.fp8_quantize_weights_new(randn((H, I), 90 + e, 0.05)) for e in range(E)]
    wu, su = torch.stack([q.view(torch.uint8) for q, _ in up]).view(F8), torch.stack([s for _, s in up])
    wd, sd = torch.stack([q.view(torch.uint8) for q, _ in down]).view(F8), torch.stack([s for _, s in down])
    T = tokens * top
    x, sx = nv.fp8_quantize_new(X[order // top])
    gu = torch.empty((T, 2 * I), dtype=BF16, device="cuda")
    nv.fp8_gemm_grouped(x, sx, wu, su, offsets, gu)
    q, s = nv.fp8_quantize_new(gu, gated=True)
    y = torch.empty((T, H), dtype=BF16, device="cuda")
    nv.fp8_gemm_grouped(q, s, wd, sd, offsets, y)
    ends = offsets.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        check_product(gu[a:b], values(x[a:b], sx[a:b], 1), values(wu[e], su[e], 128), f"up {e}")
        check_product(y[a:b], values(q[a:b], s[a:b], 1), values(wd[e], sd[e], 128), f"down {e}")
    check_quantized(gu[:, :I].double() * torch.sigmoid(gu[:, :I].double()) * gu[:, I:].double(), q, s, 2.0 ** -15)


def test_bf16_norm_feeds_the_4_bit_layer(nv):
    """The norm's BF16 output through the NVFP4 GEMV, beside its 8-bit output through the 8-bit product."""
    K, N = 1024, 512
    x, w = randn((1, K), 1), randn((K,), 2)
    W = randn((N, K), 3, 0.02)
    y, q = torch.empty_like(x), torch.empty((1, K), dtype=F8, device="cuda")
    s = torch.empty((1, 8), dtype=F32, device="cuda")
    nv.fp8_rmsnorm(x, w, y=y, q=q, s=s)
    q4, s4, g = nv.quantize_new(W)
    o4, o8 = torch.empty(N, dtype=BF16, device="cuda"), torch.empty((1, N), dtype=BF16, device="cuda")
    nv.gemv(y[0], q4, s4, g, o4)
    w8, sw = nv.fp8_quantize_weights_new(W)
    nv.fp8_gemm(q, s, w8, sw, o8)
    ref = norm_ref(x, None, w, 1e-6)[1] @ W.double().T
    # half a step of E2M1 weights is at most 2^-2 of a value, of E4M3 2^-4 on both
    # sides; their errors are independent, so the outputs stay well inside these norms
    assert float((o4.double() - ref[0]).norm() / ref.norm()) < 0.25
    assert float((o8.double() - ref).norm() / ref.norm()) < 0.125
