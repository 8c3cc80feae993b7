"""mla_rms_norm_fp8 against the norm in 64 bits.

Tolerance: fp32 sums over at most 32 values a thread, ten tree steps, a
division, a square root within 2 units, and four products keep each value
within 64 * 2^-24 of itself; a code is then off by at most half an E4M3 step
of its block scale, and the block scale is that of a maximum within the same
64 * 2^-24."""
import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
REL = 64 * 2.0 ** -24


def exponent(amax):
    """Least e with amax 2^-e <= 448, at least -127; 0 for 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-127)
    return torch.where(amax == 0, 0, e)


def verify(x, res, w, eps, codes, scales, res_out):
    s = x.float() + res.float() if res is not None else x.float()
    if res_out is not None:
        assert torch.equal(res_out, s.to(x.dtype))
    s = x.double() + (res.double() if res is not None else 0.0)
    v = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps) * w.double()
    n, d = v.shape
    v = v.view(n, d // 32, 32)
    amax = v.abs().amax(-1)
    e = scales.int() - 127
    assert torch.all((e >= exponent(amax * (1 - REL))) & (e <= exponent(amax * (1 + REL))))
    z = v * torch.exp2(-e.double()).unsqueeze(-1)
    got = codes.contiguous().view(torch.float8_e4m3fn).double().view(n, d // 32, 32)
    step = torch.exp2(torch.floor(torch.log2((z.abs() * (1 + REL)).clamp_min(2.0 ** -6))) - 3)
    err = (got - z).abs()
    assert torch.all(err <= step / 2 + REL * z.abs()), float((err - step / 2 - REL * z.abs()).max())


def run(x, res, w, eps=1e-6, want_res=None, records=False):
    n, d = x.shape
    want_res = res is not None if want_res is None else want_res
    if records:
        rec = torch.full((n, d + d // 32 + 8), 0xEE, dtype=torch.uint8, device=DEV)
        codes, scales = rec[:, :d], rec[:, d:d + d // 32]
    else:
        codes = torch.full((n, d), 0xEE, dtype=torch.uint8, device=DEV)
        scales = torch.full((n, d // 32), 0xEE, dtype=torch.uint8, device=DEV)
    res_out = torch.empty_like(x) if want_res else None
    mla.rms_norm_fp8(x, w, eps, codes, scales, residual=res, residual_out=res_out)
    verify(x, res, w, eps, codes, scales, res_out)
    if records:
        assert torch.all(rec[:, d + d // 32:] == 0xEE)
    return codes, scales


def inputs(n, d, dtype, seed=0, spread=4.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, d, generator=g, device=DEV) * torch.exp(spread * torch.randn(n, 1, generator=g, device=DEV))
    w = 1.0 + 0.3 * torch.randn(d, generator=g, device=DEV)
    r = 2.0 * torch.randn(n, d, generator=g, device=DEV)
    return x.clamp(-3e4, 3e4).to(dtype), r.to(dtype), w.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 32), (3, 64), (1, 512), (9, 512), (1000, 512), (5, 288), (7, 544), (4, 1024), (6, 1056),
                                 (3, 2048), (2, 2080), (5, 4096), (3, 5120), (2, 7168), (3, 8192), (2, 8224), (3, 16384),
                                 (257, 96)])
def test_matches_64_bits(n, d, dtype):
    x, r, w = inputs(n, d, dtype, seed=n + d)
    run(x, None, w)
    run(x, r, w, eps=1e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_awkward_rows(dtype):
    x, r, w = inputs(12, 512, dtype, seed=2)
    x[0] = 0.0                       # a row of zeros: zero codes under scale 1
    x[1, :32] = 0.0                  # an all-zero block
    x[2] = 0.0
    x[2, 5] = 100.0                  # one value carries the row
    x[3] = 1.0
    w2 = w.clone()
    w2[64:96] = 0.0
    w2[100] = -w2[100]
    codes, scales = run(x, None, w2)
    assert torch.all(codes[0] & 0x7F == 0) and torch.all(scales[0] == 127) and torch.all(scales[:, 2] == 127)
    # Equal values of weight one: v = 1 / sqrt(1 + eps), the largest power-of-two range that holds it.
    run(torch.ones(2, 512, dtype=dtype, device=DEV), None, torch.ones(512, dtype=dtype, device=DEV), eps=0.0)
    run(x, r, w2, want_res=False)    # the sum is normed and dropped
    run(x, None, w2, want_res=True)  # no residual: its copy


def test_very_small_and_large_values():
    for scale, eps in ((1e-18, 0.0), (1e17, 1e-6), (2.0 ** -70, 1e-30)):
        x, _, w = inputs(4, 1024, torch.float32, seed=4, spread=0.0)
        run(x * scale, None, w, eps=eps)
    # eps far above the mean square: blocks near the bottom of the e8m0 range.
    x, _, w = inputs(4, 512, torch.float32, seed=5, spread=0.0)
    codes = torch.empty(4, 512, dtype=torch.uint8, device=DEV)
    scales = torch.empty(4, 16, dtype=torch.uint8, device=DEV)
    mla.rms_norm_fp8(x * 2.0 ** -120, w, 1.0, codes, scales)
    verify(x * 2.0 ** -120, None, w, 1.0, codes, scales, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [512, 1024, 8192, 8224])            # a warp a row, more of them, a block, the long rows
@pytest.mark.parametrize("res", [False, True])
def test_blocks_of_tiny_values_beside_zeros(dtype, d, res):
    """Blocks whose values times 1 / rms are normal numbers, though 1 / rms times the block's scale is not."""
    x = torch.full((6, d), 0.3, dtype=dtype, device=DEV)
    x[:, 32:64] = 0.0
    x[0, 40] = 1e-37                                  # scale clamped
    x[1, 32:64:3] = -4e-37
    x[2, 63] = 6e-36
    x[3:] = 0.0
    x[3, 37] = 1e-37                                  # the row's only value: 1 / rms is 1000
    x[4, 33], x[4, d - 1] = 3e-35, -2e-37
    x[5, ::2] = 7e-37
    r = torch.zeros_like(x) if res else None
    w = torch.linspace(0.5, 2.0, d, device=DEV).to(dtype)
    codes, scales = run(x, r, w)
    assert not torch.any((codes & 0x7F) == 0x7F)      # no NaN
    assert torch.all(codes[x == 0] & 0x7F == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [512, 8224])
def test_weights_whose_product_with_the_row_leaves_the_range(dtype, d):
    """s w overflows or vanishes in 32 bits, s / rms w does not."""
    x, _, w = inputs(5, d, torch.float32, seed=23, spread=0.0)
    for rows, weights, eps in ((1e15, 1e30, 1e-6), (1e-12, 1e-30, 1e-30), (1e-15, 1e-33, 0.0)):
        run((x * rows).to(dtype), None, (w * weights).to(dtype), eps=eps)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 12800), (torch.float32, 12832), (torch.float32, 16384),
                                     (torch.bfloat16, 16384)])
def test_rows_around_the_longest_that_are_copied_ahead(dtype, d):
    """Two rows with their residuals just fit into a block's shared memory, or just do not: several rows a block, blocks of
    tiny values and of zeros among them."""
    x, r, w = inputs(400, d, dtype, seed=d)
    run(x, r, w)
    r[3::5], x[3::5] = 0.0, 0.0
    x[3::5, 70] = 1e-37
    x[8::5, :64] = 0.0
    run(x, r, w)
    run(x, None, w)
    clean = run(x, r, w)
    x[7, 5] = float("nan")
    codes, scales = torch.empty_like(clean[0]), torch.empty_like(clean[1])
    mla.rms_norm_fp8(x, w, 1e-6, codes, scales, residual=r)
    keep = [i for i in range(400) if i != 7]
    assert torch.equal(codes[keep], clean[0][keep]) and torch.equal(scales[keep], clean[1][keep])


def test_a_row_of_infinities_or_nan_spoils_no_other():
    x, r, w = inputs(20, 512, torch.bfloat16, seed=6)
    clean = run(x, r, w)
    x2 = x.clone()
    x2[3, 7], x2[9, 100], x2[10, 0] = float("inf"), float("nan"), float("-inf")
    codes = torch.empty(20, 512, dtype=torch.uint8, device=DEV)
    scales = torch.empty(20, 16, dtype=torch.uint8, device=DEV)
    mla.rms_norm_fp8(x2, w, 1e-6, codes, scales, residual=r)
    keep = [i for i in range(20) if i not in (3, 9, 10)]
    assert torch.equal(codes[keep], clean[0][keep]) and torch.equal(scales[keep], clean[1][keep])


def test_cache_records_strided_inputs_and_in_place_residual():
    x, r, w = inputs(33, 512, torch.bfloat16, seed=7)
    run(x, r, w, records=True)
    wide = torch.randn(33, 1536, device=DEV).to(torch.bfloat16)
    xs, rs = wide[:, 512:1024], wide[:, 1024:]
    codes, scales = run(xs, rs, w)
    before = wide.clone()
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    mla.rms_norm_fp8(xs, w, 1e-6, c2, s2, residual=rs, residual_out=rs)       # the stream is updated where it lies
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    assert torch.equal(wide[:, 1024:], (before[:, 512:1024].float() + before[:, 1024:].float()).to(torch.bfloat16))
    assert torch.equal(wide[:, :1024], before[:, :1024])
    # One broadcast row as the residual (stride 0) and as the input.
    run(x[:1].expand(33, 512), r[:1].expand(33, 512), w, want_res=True)


def test_records_dequantize_as_the_cache_reads_them():
    x, _, w = inputs(64, 512, torch.bfloat16, seed=8, spread=0.5)
    rec = torch.empty(64, 528, dtype=torch.uint8, device=DEV)
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.rms_norm_fp8(x, w, 1e-6, rec[:, :512], rec[:, 512:], error=error)
    assert int(error) == 0
    got = mla.dequantize(rec).double()
    v = x.double()
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    amax = v.view(64, 16, 32).abs().amax(-1, keepdim=True)
    # Half an E4M3 step: 2^-4 of the value, or 2^-10 of the scale for small ones (scale < amax / 224 (1 + REL)).
    tol = torch.maximum(v.view(64, 16, 32).abs() / 16, amax / 224 * 2.0 ** -10 * (1 + 2 * REL))
    assert torch.all((got.view(64, 16, 32) - v.view(64, 16, 32)).abs() <= tol + REL * amax)


def test_streams_graphs_and_refusals():
    x, r, w = inputs(40, 512, torch.bfloat16, seed=9)
    codes = torch.zeros(40, 512, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(40, 16, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    mla.rms_norm_fp8(x, w, 1e-6, codes, scales, residual=r, residual_out=out, stream=s)
    s.synchronize()
    verify(x, r, w, 1e-6, codes, scales, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mla.rms_norm_fp8(x, w, 1e-6, codes, scales, residual=r, residual_out=out)
    x.normal_()
    g.replay()
    torch.cuda.synchronize()
    verify(x, r, w, 1e-6, codes, scales, out)
    mla.rms_norm_fp8(x[:0], w, 1e-6, codes[:0], scales[:0])
    with pytest.raises(ValueError):
        mla.rms_norm_fp8(x, w.float(), 1e-6, codes, scales)
    with pytest.raises(ValueError):
        mla.rms_norm_fp8(x, w, 1e-6, codes[:, :256], scales)
    with pytest.raises(ValueError):
        mla.rms_norm_fp8(x, w, 1e-6, codes, scales.view(torch.int8))
    with pytest.raises(mla.MLAError):
        mla.rms_norm_fp8(x[:, 1:481], w[1:481].clone(), 1e-6, codes[:, :480], scales[:, :15])   # rows off 16 bytes


@pytest.mark.parametrize("d", [512, 8224])
def test_offsets_beyond_32_bits(d):
    """Rows whose element offsets pass 2^31 (4.8 GB of bf16, of which little is touched)."""
    wide = torch.empty(600, 1 << 22, dtype=torch.bfloat16, device=DEV)
    x, r, w = inputs(600, d, torch.bfloat16, seed=22)
    a, b = wide[:, 64:64 + d], wide[:, 1 << 20:(1 << 20) + d]
    a.copy_(x)
    b.copy_(r)
    codes = torch.empty(600, d, dtype=torch.uint8, device=DEV)
    scales = torch.empty(600, d // 32, dtype=torch.uint8, device=DEV)
    mla.rms_norm_fp8(a, w, 1e-6, codes, scales, residual=b, residual_out=b)
    verify(x, r, w, 1e-6, codes, scales, b)
