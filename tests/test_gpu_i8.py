"""The 8-bit linear path and the query/key norm with rotation against their definitions in 64 bits.

u = 2^-24 is FP32's half step; a BF16 rounding is off by at most 2^-8 of the value.  The bounds are
written beside each reference; none is fitted to what the kernels give.
"""
import ctypes
import subprocess
import sys

import numpy as np
import pytest
import torch

import diffusion_transformer_text_block_b200 as moss
from oracle import moss_oracle as o
from tests.conftest import ROOT
from tests.gpu_common import assert_no_device_error

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert_no_device_error()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen(seed), device="cuda") * scale


def ints(seed, *shape):
    return torch.randint(-127, 128, shape, generator=gen(seed), device="cuda", dtype=torch.int8)


# ------------------------------------------------------------------------------ rows to 8 bits
def quantized(h):
    """(q, scale) of float64 rows by the definition; torch.round takes halves to even.  127 h is exact for
    an FP32 h, and a quotient that is no half-integer stays 2^-34 away from one, far above FP64's rounding."""
    amax = h.abs().amax(dim=1, keepdim=True)
    q = torch.round(h * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q, (amax / 127.0)[:, 0]


def check_scale(scale, ref):
    """One correctly rounded FP32 division (2^-150: half of the smallest subnormal step)."""
    assert ((scale.double() - ref).abs() <= U * ref + 2.0 ** -150).all()


ROWS_DIMS = [(1, 16), (3, 64), (2, 48), (37, 704), (33, 256), (1, 3072), (333, 3072), (77, 4096), (5, 8192), (7, 32768),
             (2, 20000), (1201, 1040)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", ROWS_DIMS)
def test_quantize_is_exact(rows, dim, dtype):
    x = (randn(1, rows, dim) * torch.exp(randn(2, rows, 1))).to(dtype)
    x[rows // 2] = 0
    q, scale = moss.op_quantize_i8(x)
    ref, ref_scale = quantized(x.double())
    assert torch.equal(q.double(), ref)
    check_scale(scale, ref_scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_halves(dtype):
    """Rows made of exact halves of a step and of values next to them: amax 254 * 2^e puts the steps at
    2^(e+1), so odd multiples of 2^e lie on a border and go to the even side."""
    steps = torch.arange(-254, 255, device="cuda", dtype=torch.float64)
    base = torch.cat([steps, steps[:3]])  # 512 values
    rows = [base * 2.0 ** e for e in (-140, -126, -100, -20, 0, 7, 100, 119)]
    x = torch.stack(rows).to(dtype)
    inf = torch.tensor(float("inf"), device="cuda")
    for v in (x, torch.nextafter(x, inf), torch.nextafter(x, -inf)) if dtype == torch.float32 else (x,):
        q, scale = moss.op_quantize_i8(v)
        ref, ref_scale = quantized(v.double())
        assert torch.equal(q.double(), ref)
        check_scale(scale, ref_scale)


@pytest.mark.parametrize("e", [0, -50, -126, 112])
def test_quantize_every_ratio_of_bf16_values(e):
    """Every significand of the largest element against every significand of the others down to 2^-10 of it:
    the rule that BF16 rows are rounded without a check holds for all of them."""
    sig = torch.arange(128, 256, dtype=torch.float64, device="cuda")
    amax = sig[:, None] * 2.0 ** e
    others = torch.cat([sig * 2.0 ** (e - i) for i in range(11)])[None, :]
    x = torch.where(others <= amax, others, torch.zeros_like(others))
    x = torch.cat([amax, x, -x, torch.zeros(128, 15, dtype=torch.float64, device="cuda")], dim=1)
    xb = x.to(torch.bfloat16)
    assert torch.equal(xb.double(), x) or e < -100
    q, scale = moss.op_quantize_i8(xb)
    ref, ref_scale = quantized(xb.double())
    assert torch.equal(q.double(), ref)
    check_scale(scale, ref_scale)


@pytest.mark.parametrize("dim", [256, 768, 1024, 1536, 2048, 3072, 4096, 6144, 8192, 12288, 16384])
@pytest.mark.parametrize("rows", [2, 200, 700, 1300])
def test_every_team_size(rows, dim):
    """Rows that fill their lanes exactly, with 1, 2, 4 and 8 warps a row as the number of rows asks for: all
    four sources, the integers exact for BF16 and FP32 rows and within FP32's error of h for the others."""
    x = randn(11, rows, dim)
    for v in (x, x.bfloat16()):
        q, scale = moss.op_quantize_i8(v)
        ref, ref_scale = quantized(v.double())
        assert torch.equal(q.double(), ref)
        check_scale(scale, ref_scale)
    shift, mscale = randn(12, dim, scale=0.1), randn(13, dim, scale=0.1)
    q, qs = moss.op_ln_modulate_i8(x, shift, mscale)
    check_rows_of(q, qs, *layer_norm_reference(x, shift, mscale))
    gu = randn(14, rows, 2 * dim, scale=2.0).bfloat16()
    q, qs = moss.op_swiglu_i8(gu)
    check_rows_of(q, qs, *swiglu_reference(gu))


def test_quantize_extremes():
    """Subnormal rows, the largest finite values, one element set, and rows that are not finite."""
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    x = torch.zeros(9, 64, device="cuda")
    x[0, 3] = tiny
    x[1, :4] = torch.tensor([tiny, 2 * tiny, 3 * tiny, -5 * tiny], device="cuda")
    x[2] = randn(3, 64) * 1e-39
    x[3] = randn(4, 64) * 1e-31
    x[4] = randn(5, 64) * (big / 8)
    x[5, :2] = torch.tensor([big, -big / 2], device="cuda")
    x[6, 7] = float("inf")
    x[7, 9] = float("nan")
    x[8] = -2.0 ** -100
    q, scale = moss.op_quantize_i8(x)
    fine = [0, 1, 2, 3, 4, 5, 8]
    ref, ref_scale = quantized(x.double())
    assert torch.equal(q[fine].double(), ref[fine])
    check_scale(scale[fine], ref_scale[fine])
    assert torch.isnan(scale[6:8]).all() and (q[6:8] == 0).all()


def test_rows_with_a_stride_and_their_surroundings():
    """Rows inside wider ones; what lies before, between and behind the outputs' rows stays as it was."""
    wide = randn(6, 21, 3 * 704).bfloat16()
    x = wide[2:20, 704:1408]
    q, scale = moss.op_quantize_i8(x)
    q2, scale2 = moss.op_quantize_i8(x.contiguous())
    assert torch.equal(q, q2) and torch.equal(scale, scale2)
    gu = wide[1:19, 704:]
    a, b = moss.op_swiglu_i8(gu), moss.op_swiglu_i8(gu.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    buf = torch.full((5, 704), 99, device="cuda", dtype=torch.int8)
    sbuf = torch.full((16,), -7.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    for rows in (1, 3):
        rc = moss.lib().moss_op_quantize_i8(x.data_ptr(), moss.DTYPE_BF16, 3 * 704, buf[1].data_ptr(), sbuf[4:].data_ptr(),
                                            rows, 704, s)
        assert rc == 0
        assert (buf[0] == 99).all() and (buf[1 + rows:] == 99).all() and torch.equal(buf[1:1 + rows], q[:rows])
        assert (sbuf[:4] == -7).all() and (sbuf[4 + rows:] == -7).all()


def check_rows_of(q, scale, h, err):
    """q * scale against h (float64), where the kernel's FP32 rows are within err of h: an element is off by
    its own error, half a step (of a scale that the largest error moved) and FP32's roundings of 127 / amax
    and of the scale, u of the element each."""
    amax = h.abs().amax(dim=1)
    emax = err.amax(dim=1)
    assert ((scale.double() - amax / 127).abs() <= emax / 127 + 2 * U * amax / 127).all()
    bound = err + (0.5 * (amax / 127 + emax / 127) + 2 * U * amax + U * emax)[:, None]
    assert ((q.double() * scale.double()[:, None] - h).abs() <= bound).all()


def layer_norm_reference(x, shift, scale):
    """(h, bound on FP32's error).  A sum of at most 16 x 8 terms a lane, 5 shuffles and 8 warps is off by
    d u sum|x| with d = 141; the centred value x - mean by d u mean|x| + u|x - mean|; the variance, a sum
    of squares of those, relatively by (d + 4) u + 2 d u mean|x| / std (first order), 1/std by half of that and
    rsqrtf's 2 ulp (4 u); (1 + scale), the product and the sum add 4 u."""
    xd, m = x.double(), 1 + scale.double()
    mean = xd.mean(dim=1, keepdim=True)
    std = torch.sqrt(((xd - mean) ** 2).mean(dim=1, keepdim=True) + 1e-6)
    n = (xd - mean) / std
    h = n * m + shift.double()
    d, mabs = 141, xd.abs().mean(dim=1, keepdim=True)
    err = m.abs() * ((d * U * mabs / std) + n.abs() * U * (1 + (d + 4) / 2 + d * mabs / std + 4 + 4)) + 2 * U * h.abs()
    return h, 1.01 * err


def swiglu_reference(gu):
    """(h, bound on FP32's error).  h = g / (1 + e^-g) u: __expf is within 2 + 1.173|g| ulp (2 u each), which the
    sum weakens; the sum, the approximate division (2 ulp) and the product add 1 + 4 + 1 u."""
    g, u = gu.double().chunk(2, dim=1)
    h = g * torch.sigmoid(g) * u
    return h, 1.01 * h.abs() * U * (2 * (2 + 1.173 * g.abs()) + 8)


@pytest.mark.parametrize("rows,dim", [(1, 128), (37, 256), (333, 3072), (5, 8192), (2, 20000), (1, 16)])
def test_ln_modulate_i8(rows, dim):
    x = randn(7, rows, dim, scale=3.0) + 0.5
    shift, scale = randn(8, dim, scale=0.1), randn(9, dim, scale=0.1)
    q, qs = moss.op_ln_modulate_i8(x, shift, scale)
    h, err = layer_norm_reference(x, shift, scale)
    ref = torch.from_numpy(o.ln_modulate(x.double().cpu().numpy(), shift.double().cpu().numpy(), scale.double().cpu().numpy()))
    assert (h.cpu() - ref).abs().max() <= 1e-12
    check_rows_of(q, qs, h, err)


@pytest.mark.parametrize("rows,dim", [(1, 64), (37, 704), (333, 8192), (2, 32768), (3, 16)])
def test_swiglu_i8(rows, dim):
    gu = randn(10, rows, 2 * dim, scale=2.0).bfloat16()
    gu[:, 0], gu[:, 1], gu[:, dim:dim + 2] = -40.0, 30.0, 0.5
    q, qs = moss.op_swiglu_i8(gu)
    check_rows_of(q, qs, *swiglu_reference(gu))


def test_swiglu_limits():
    """A gate far below zero gives 0, one far above passes; what is not finite marks its row."""
    gu = torch.ones(4, 32, device="cuda", dtype=torch.bfloat16)
    gu[0, :4] = torch.tensor([-88.0, -100.0, -1e4, 200.0])
    gu[1, 20] = float("inf")
    gu[2, 3] = float("nan")
    gu[3] = 0
    q, qs = moss.op_swiglu_i8(gu)
    assert q[0, :4].tolist() == [0, 0, 0, 127] and abs(float(qs[0]) - 200 / 127) < 1e-5
    assert torch.isnan(qs[1:3]).all() and (q[1:3] == 0).all()
    assert float(qs[3]) == 0 and (q[3] == 0).all()


# ------------------------------------------------------------------------------ the 8-bit GEMM
def gemm_case(seed, M, N, K, bias, resid):
    a, b = ints(seed, M, K), ints(seed + 1, N, K)
    sa, sb = torch.rand(M, generator=gen(seed + 2), device="cuda") + 0.01, torch.rand(N, generator=gen(seed + 3), device="cuda") * 1e-3
    bi = randn(seed + 4, N).bfloat16() if bias else None
    gate = randn(seed + 5, N) if resid else None
    res = randn(seed + 6, M, N, scale=30.0) if resid else None
    return a, sa, b, sb, bi, gate, res


def check_gemm(c, a, sa, b, sb, bias, gate, res, rows=None):
    """Per element: the sum is exact; its rounding to FP32, two scales and the bias cost 4 u of the terms,
    the gate and the residual 2 u more, and BF16 2^-8 of the result."""
    if rows is not None:
        a, sa, c = a[rows], sa[rows], c[rows]
        res = res[rows] if res is not None else None
    ref = (a.double() @ b.double().T) * sa.double()[:, None] * sb.double()
    mag = ref.abs()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    if res is not None:
        ref, mag = res.double() + gate.double() * ref, res.double().abs() + gate.double().abs() * mag
    bound = 6.1 * U * mag + (BF * (ref.abs() + 6.1 * U * mag) if c.dtype == torch.bfloat16 else 0)
    assert ((c.double() - ref).abs() <= bound).all(), ((c.double() - ref).abs() - bound).max()


GEMM_SIZES = [(1, 1, 16), (1, 128, 64), (1, 9216, 3072), (2, 7, 48), (15, 96, 128), (16, 129, 144), (17, 127, 256),
              (33, 300, 704), (64, 704, 256), (65, 257, 1040), (77, 3072, 4096), (128, 384, 8192), (129, 131, 272),
              (255, 513, 320), (256, 256, 640), (257, 255, 3072), (300, 1000, 4096), (513, 704, 256), (1024, 768, 3072),
              (2304, 3072, 1024), (4429, 1024, 256), (3, 2, 65536), (9, 8200, 64), (16, 8192, 80),
              (20, 20000, 256), (100, 19001, 128), (20001, 300, 16),
              (50001, 1, 64), (17, 1, 16), (8, 5, 8192), (11, 33, 4096), (16, 40, 16384)]


@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
@pytest.mark.parametrize("form", ["bf16", "f32", "bias", "resid"])
def test_gemm(M, N, K, form):
    args = gemm_case(20, M, N, K, form in ("bias", "resid"), form == "resid")
    a, sa, b, sb, bias, gate, res = args
    c = moss.op_gemm_i8(a, sa, b, sb, bias=bias, gate=gate, residual=res,
                        out_dtype=torch.float32 if form in ("f32", "resid") else torch.bfloat16)
    check_gemm(c, *args)


def test_gemm_sums_are_exact():
    """The largest sums: 2^30 in every element (and -2^30 + 2^23 with 127), as scale 1 shows them."""
    for M, N in ((2, 130), (300, 300)):
        one = torch.ones(max(M, N), device="cuda")
        a = torch.full((M, 65536), -128, device="cuda", dtype=torch.int8)
        b = torch.full((N, 65536), -128, device="cuda", dtype=torch.int8)
        b[N // 2:] = 127
        c = moss.op_gemm_i8(a, one[:M].contiguous(), b, one[:N].contiguous(), out_dtype=torch.float32)
        assert (c[:, :N // 2] == 2.0 ** 30).all() and (c[:, N // 2:] == -128.0 * 127 * 65536).all()


def test_gemm_in_place_and_surroundings():
    M, N, K = 77, 704, 256
    a, sa, b, sb, bias, gate, res = gemm_case(30, M, N, K, True, True)
    want = moss.op_gemm_i8(a, sa, b, sb, bias=bias, gate=gate, residual=res)
    buf = torch.full((M + 2, N), -3.0, device="cuda")
    buf[1:M + 1] = res
    got = moss.op_gemm_i8(a, sa, b, sb, bias=bias, gate=gate, residual=buf[1:M + 1], out=buf[1:M + 1])
    assert torch.equal(got, want) and (buf[0] == -3).all() and (buf[M + 1] == -3).all()
    for M2 in (1, 5, 16, 40, 76):
        out = torch.full((M + 1, N), 5.0, device="cuda", dtype=torch.bfloat16)
        moss.op_gemm_i8(a[:M2], sa[:M2], b, sb, out=out[:M2])
        assert (out[M2:] == 5).all()
        check_gemm(out[:M2], a[:M2], sa[:M2], b, sb, None, None, None)


def test_gemm_scales_that_are_not_finite_stay_in_their_row_and_column():
    a, sa, b, sb, *_ = gemm_case(40, 40, 200, 128, False, False)
    sa[3], sb[150] = float("nan"), float("inf")
    sa[7] = 0.0
    c = moss.op_gemm_i8(a, sa, b, sb, out_dtype=torch.float32)
    assert torch.isnan(c[3]).all()
    keep = [i for i in range(40) if i != 3]
    cols = [j for j in range(200) if j != 150]
    assert torch.isfinite(c[keep][:, cols]).all() and (c[7][cols] == 0).all()
    assert not torch.isfinite(c[keep, 150]).any()


def test_gemm_output_beyond_32_bit_offsets():
    """70001 x 32768 outputs: element offsets pass 2^31; rows at the ends, the middle and the border."""
    M, N, K = 70001, 32768, 64
    a, sa, b, sb, *_ = gemm_case(50, M, N, K, False, False)
    c = moss.op_gemm_i8(a, sa, b, sb)
    rows = torch.tensor([0, 1, 65535, 65536, 65537, 69999, 70000, 35000], device="cuda")
    check_gemm(c, a, sa, b, sb, None, None, None, rows=rows)


def test_calls_from_two_threads():
    """Two threads, a stream each, calls of different kernels: nothing is shared but what the library guards."""
    import threading
    cases = [gemm_case(62, 300, 704, 1024, False, False), gemm_case(72, 5, 3072, 1024, False, False)]
    want = [moss.op_gemm_i8(*c[:4]) for c in cases]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i].append(moss.op_gemm_i8(*cases[i][:4]))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (0, 1):
        assert len(got[i]) == 50 and all(torch.equal(g, want[i]) for g in got[i])


def test_gemm_is_the_same_on_two_streams_at_once():
    one, two = gemm_case(60, 300, 704, 1024, False, False), gemm_case(70, 5, 3072, 1024, True, False)
    w1 = moss.op_gemm_i8(*one[:4])
    w2 = moss.op_gemm_i8(*two[:4], bias=two[4])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        with torch.cuda.stream(s1):
            got.append((moss.op_gemm_i8(*one[:4]), w1))
        with torch.cuda.stream(s2):
            got.append((moss.op_gemm_i8(*two[:4], bias=two[4]), w2))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in got)


def test_a_stream_given_by_name_or_handle():
    """The call runs on it, and its new tensors come from its pool: a long kernel before it on the current
    stream holds nothing up and no memory of that stream is taken."""
    a, sa, b, sb, bias, *_ = gemm_case(75, 40, 704, 512, True, False)
    x = randn(76, 40, 512)
    want = moss.op_gemm_i8(a, sa, b, sb, bias=bias), moss.op_quantize_i8(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream, torch.cuda.default_stream(), 0):
        got = moss.op_gemm_i8(a, sa, b, sb, bias=bias, stream=given), moss.op_quantize_i8(x, stream=given)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and all(torch.equal(g, w) for g, w in zip(got[1], want[1]))


# ------------------------------------------------------------------------------ query/key norm and rotation
def qk_reference(x, gain, rope, pos, pairing, eps):
    """(y, bound on FP32's error) of [rows, heads, d]: the sum of squares (13 additions of positive terms), the
    mean and rsqrtf leave 1/rms within (15 / 2 + 4) u; the product with it, gain * cos, the two products of a
    pair and their sum add 5 u: 16.5 u of the pair's terms."""
    x = x.double()
    n = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    if gain is not None:
        n = n * gain.double()
    y, mag = n.clone(), n.abs()
    if rope is not None:
        r = 2 * rope.shape[1]
        cos, sin = rope[pos][:, None, :, 0].double(), rope[pos][:, None, :, 1].double()
        ia = torch.arange(0, r, 2) if pairing == "adjacent" else torch.arange(0, r // 2)
        ib = ia + 1 if pairing == "adjacent" else ia + r // 2
        a, b = n[..., ia], n[..., ib]
        y[..., ia], y[..., ib] = a * cos - b * sin, a * sin + b * cos
        mag[..., ia] = (a * cos).abs() + (b * sin).abs()
        mag[..., ib] = (a * sin).abs() + (b * cos).abs()
    return y, 17 * U * mag


def check_qk(got, x, gain, rope, pos, pairing, eps):
    y, err = qk_reference(x, gain, rope, pos, pairing, eps)
    bound = err + (BF * (y.abs() + err) if got.dtype == torch.bfloat16 else U * y.abs())
    assert ((got.double() - y).abs() <= bound + 1e-38).all(), ((got.double() - y).abs() - bound).max()


def angles(seed, npos, rot):
    t = torch.rand(npos, rot // 2, generator=gen(seed), device="cuda", dtype=torch.float64) * 6.4
    return torch.stack([torch.cos(t), torch.sin(t)], dim=-1).float().contiguous()


@pytest.mark.parametrize("rows,hq,hk,d,rot,pairing", [
    (1, 1, 0, 128, 128, "adjacent"), (1, 24, 24, 128, 128, "adjacent"), (8, 32, 8, 128, 128, "halves"),
    (333, 24, 24, 128, 128, "adjacent"), (1000, 5, 3, 128, 128, "halves"), (5, 3, 1, 64, 64, "halves"),
    (1, 7, 7, 64, 32, "adjacent"), (77, 16, 2, 64, 40, "halves"), (3, 4, 1, 256, 64, "halves"),
    (130, 9, 3, 256, 256, "adjacent"), (9, 2, 2, 128, 8, "halves"), (4, 40, 8, 128, 0, "adjacent"),
    (2049, 3, 3, 256, 128, "halves")])
@pytest.mark.parametrize("tin,tout", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                      (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
def test_qk_norm_rope(rows, hq, hk, d, rot, pairing, tin, tout):
    width = (hq + 2 * hk) * d
    qkv = (randn(80, rows, width) * torch.exp(randn(81, rows, 1))).to(tin)
    qkv[rows // 2] = 0
    before = qkv.clone()
    q, k = qkv[:, :hq * d].view(rows, hq, d), qkv[:, hq * d:(hq + hk) * d].view(rows, hk, d)
    gq, gk = 1 + randn(82, d, scale=0.1), 1 + randn(83, d, scale=0.1)
    npos = 19
    rope = angles(84, npos, rot) if rot else None
    for given in (False, True):
        if given and rope is None:
            continue
        pos = torch.randint(0, npos, (rows,), generator=gen(85), device="cuda", dtype=torch.int32) if given else None
        at = pos.long() if given else torch.arange(rows, device="cuda") % npos
        qo, ko = moss.op_qk_norm_rope(q, k if hk else None, gq, gk if hk else None, rope, positions=pos, pairing=pairing,
                                      out_dtype=tout)
        check_qk(qo, q, gq, rope, at, pairing, 1e-6)
        if hk:
            check_qk(ko, k, gk, rope, at, pairing, 1e-6)
        assert torch.equal(qkv, before)


def test_qk_in_place_leaves_the_values_and_matches_out_of_place():
    rows, H, d = 77, 3, 128
    qkv = randn(90, rows + 1, 3 * H * d).bfloat16()
    start = qkv.clone()
    q, k = qkv[:rows, :H * d].view(rows, H, d), qkv[:rows, H * d:2 * H * d].view(rows, H, d)
    gain, rope = 1 + randn(91, d, scale=0.1), angles(92, rows, d)
    want = moss.op_qk_norm_rope(q, k, gain, gain, rope)
    moss.op_qk_norm_rope(q, k, gain, gain, rope, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, 2 * H * d:], start[:, 2 * H * d:]) and torch.equal(qkv[rows], start[rows])


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_qk_from_and_to_buffers_of_other_strides(pairing):
    """q and k in tensors of their own, written into the columns of a wider buffer."""
    rows, hq, hk, d = 45, 6, 2, 64
    q, k = randn(86, rows + 3, hq + 1, d)[:rows, :hq], randn(87, rows, hk, d)
    gq, gk, rope = 1 + randn(88, d, scale=0.1), 1 + randn(89, d, scale=0.1), angles(90, rows, d)
    wide = torch.full((rows, 3 * d + (hq + hk) * d + d), 4.0, device="cuda", dtype=torch.bfloat16)
    qo = wide[:, 2 * d:(2 + hq) * d].view(rows, hq, d)
    ko = wide[:, (3 + hq) * d:(3 + hq + hk) * d].view(rows, hk, d)
    moss.op_qk_norm_rope(q, k, gq, gk, rope, pairing=pairing, q_out=qo, k_out=ko)
    at = torch.arange(rows, device="cuda")
    check_qk(qo, q, gq, rope, at, pairing, 1e-6)
    check_qk(ko, k, gk, rope, at, pairing, 1e-6)
    assert (wide[:, :2 * d] == 4).all() and (wide[:, (2 + hq) * d:(3 + hq) * d] == 4).all() and (wide[:, -d:] == 4).all()


def test_qk_without_gains_and_with_rows_that_are_not_finite():
    q = randn(93, 6, 2, 128)
    q[1, 0, 5], q[2, 1, 127] = float("nan"), float("inf")
    rope = angles(94, 6, 128)
    qo, _ = moss.op_qk_norm_rope(q, None, None, None, rope, out_dtype=torch.float32)
    bad = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert torch.isfinite(qo[~bad]).all() and torch.isnan(qo[1, 0]).any() and torch.isnan(qo[2, 1]).any()
    good = q.clone()
    good[bad] = 1.0
    y, err = qk_reference(good, None, rope, torch.arange(6, device="cuda"), "adjacent", 1e-6)
    assert (((qo.double() - y).abs() <= err + U * y.abs()) | bad[:, :, None]).all()


def test_qk_position_outside_the_table_is_left_out_and_reported():
    q = randn(95, 5, 4, 128).bfloat16()
    rope = angles(96, 8, 128)
    pos = torch.tensor([3, -1, 7, 8, 0], device="cuda", dtype=torch.int32)
    out = torch.full((5, 4, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    moss.op_qk_norm_rope(q, None, None, None, rope, positions=pos, q_out=out)
    torch.cuda.synchronize()
    assert moss.device_status(clear=True) == 0x401
    keep = torch.tensor([0, 2, 4], device="cuda")
    assert (out[[1, 3]] == 9).all()
    check_qk(out[keep], q[keep], None, rope, pos[keep].long(), "adjacent", 1e-6)


def test_qk_beyond_32_bit_offsets():
    """A fused buffer of 2.4e9 elements: rows at its end, through the stride."""
    rows, H, d = 262145, 24, 128
    stride = 3 * H * d
    qkv = torch.empty(rows, stride, device="cuda", dtype=torch.bfloat16)
    part = randn(97, 64, stride).bfloat16()
    for at in (0, 131072, rows - 64):
        qkv[at:at + 64] = part
    qkv[64:131072] = 1
    qkv[131136:rows - 64] = 1
    q, k = qkv[:, :H * d].view(rows, H, d), qkv[:, H * d:2 * H * d].view(rows, H, d)
    gain, rope = 1 + randn(98, d, scale=0.1), angles(99, 4608, d)
    moss.op_qk_norm_rope(q, k, gain, gain, rope, q_out=q, k_out=k)
    for at in (0, 131072, rows - 64):
        pos = (at + torch.arange(64, device="cuda")) % 4608
        check_qk(q[at:at + 64], part[:, :H * d].view(64, H, d), gain, rope, pos, "adjacent", 1e-6)
        check_qk(k[at:at + 64], part[:, H * d:2 * H * d].view(64, H, d), gain, rope, pos, "adjacent", 1e-6)


@pytest.mark.parametrize("gh,gw,nt", [(4, 6, 5), (1, 1, 0), (0, 0, 3), (64, 64, 512)])
def test_rope_table_matches_the_oracle(gh, gw, nt):
    """Angles in FP64, each (cos, sin) rounded to FP32 once."""
    t = moss.op_rope_table(gh, gw, nt).cpu().double().numpy()
    ang = o.rope_angles(o.token_positions(gh, gw, nt))
    assert np.abs(t[..., 0] - np.cos(ang)).max() <= 2.0 ** -24 and np.abs(t[..., 1] - np.sin(ang)).max() <= 2.0 ** -24


# ------------------------------------------------------------------------------ together
def block_8bit(x, w, H, rope, mod, resid_out):
    """One joint block on 8-bit products, as the header lists it; returns every step's output."""
    B, N, D = x.shape
    F = w["down"][0].shape[1]
    xf = x.view(B * N, D)
    s1, c1, g1, s2, c2, g2 = mod
    st = {}
    st["h1"] = moss.op_ln_modulate_i8(xf, s1, c1)
    qkv = moss.op_gemm_i8(*st["h1"], *w["qkv"])
    st["qkv"] = qkv.clone()
    q, k = qkv[:, :D].view(B * N, H, 128), qkv[:, D:2 * D].view(B * N, H, 128)
    moss.op_qk_norm_rope(q, k, w["qg"], w["kg"], rope, q_out=q, k_out=k)
    st["turned"] = qkv
    st["attn"] = moss.op_attention(qkv.view(B, N, 3 * D), H).view(B * N, D)
    st["attn8"] = moss.op_quantize_i8(st["attn"])
    st["mid"] = moss.op_gemm_i8(*st["attn8"], *w["o"], gate=g1, residual=xf)
    st["h2"] = moss.op_ln_modulate_i8(st["mid"], s2, c2)
    st["gu"] = moss.op_gemm_i8(*st["h2"], *w["gu"])
    st["act"] = moss.op_swiglu_i8(st["gu"])
    st["out"] = moss.op_gemm_i8(*st["act"], *w["down"], gate=g2, residual=st["mid"], out=resid_out)
    assert F == st["act"][0].shape[1]
    return st


def block_case(seed, B, gh, gw, nt, D, F):
    N = gh * gw + nt
    g = lambda i, *s, scale=1.0: randn(seed + i, *s, scale=scale)  # noqa: E731
    w = {name: moss.op_quantize_i8(g(i, *shape, scale=0.02)) for i, (name, shape) in enumerate(
        {"qkv": (3 * D, D), "o": (D, D), "gu": (2 * F, D), "down": (D, F)}.items())}
    w["qg"], w["kg"] = 1 + g(10, 128, scale=0.02), 1 + g(11, 128, scale=0.02)
    mod = [g(20 + i, D, scale=0.2) for i in range(6)]
    return g(30, B, N, D), w, moss.op_rope_table(gh, gw, nt), mod


@pytest.mark.parametrize("B,gh,gw,nt,D,F", [(2, 4, 5, 7, 256, 704), (1, 1, 1, 0, 128, 64), (1, 16, 16, 77, 1024, 2752)])
def test_block_of_8bit_operators(B, gh, gw, nt, D, F):
    """A joint block's run: each step against 64 bits on the run's own inputs to it."""
    H = D // 128
    x, w, rope, mod = block_case(100, B, gh, gw, nt, D, F)
    N = gh * gw + nt
    start = x.clone()
    out = torch.empty(B * N, D, device="cuda")
    st = block_8bit(x, w, H, rope, mod, out)
    assert torch.equal(x, start)
    check_gemm(st["qkv"], *st["h1"], *w["qkv"], None, None, None)
    pos = torch.arange(B * N, device="cuda") % N
    for i, gain in ((0, w["qg"]), (1, w["kg"])):
        cols = slice(i * D, (i + 1) * D)
        check_qk(st["turned"][:, cols].view(B * N, H, 128), st["qkv"][:, cols].view(B * N, H, 128), gain, rope, pos,
                 "adjacent", 1e-6)
    assert torch.equal(st["turned"][:, 2 * D:], st["qkv"][:, 2 * D:])
    ref, ref_scale = quantized(st["attn"].double())
    assert torch.equal(st["attn8"][0].double(), ref)
    check_gemm(st["mid"], *st["attn8"], *w["o"], None, mod[2], x.view(B * N, D))
    check_gemm(st["gu"], *st["h2"], *w["gu"], None, None, None)
    check_gemm(st["out"], *st["act"], *w["down"], None, mod[5], st["mid"])
    assert torch.isfinite(st["out"]).all()


def test_block_of_8bit_operators_captured_in_a_graph():
    """Captured once, replayed on new inputs in the same buffers: bit for bit the eager run's result."""
    x, w, rope, mod = block_case(200, 2, 4, 5, 7, 256, 704)
    out = torch.empty(2 * 27, 256, device="cuda")
    block_8bit(x, w, 2, rope, mod, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        block_8bit(x, w, 2, rope, mod, out)
    for seed in (301, 302):
        x.copy_(randn(seed, *x.shape))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = torch.empty_like(out)
        block_8bit(x, w, 2, rope, mod, want)
        assert torch.equal(got, want)


def test_first_call_of_a_process_may_be_captured():
    """The library's lazily made state (error word, kernel attributes) is set up inside a capture too."""
    code = """
import torch, diffusion_transformer_text_block_b200 as moss
a = torch.ones(5, 64, device="cuda", dtype=torch.int8); s = torch.ones(5, device="cuda")
x = torch.ones(5, 1, 128, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c = moss.op_gemm_i8(a, s, a, s, out_dtype=torch.float32)
    y, _ = moss.op_qk_norm_rope(x, None, None, None, None, out_dtype=torch.float32)
g.replay(); torch.cuda.synchronize()
assert (c == 64).all() and (y - 1).abs().max() < 1e-6 and moss.device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_binding_refusals():
    x = randn(400, 4, 64)
    i8, s = ints(401, 4, 64), torch.ones(4, device="cuda")
    for call, what in ((lambda: moss.op_quantize_i8(x.half()), "bfloat16 or torch.float32"),
                       (lambda: moss.op_quantize_i8(x.T), "contiguous rows"),
                       (lambda: moss.op_quantize_i8(x[:, 1:49]), "16-byte aligned|multiple of 16"),
                       (lambda: moss.op_quantize_i8(x[:, :40].contiguous()), "multiple of 16"),
                       (lambda: moss.op_ln_modulate_i8(x, x[0, :32].contiguous(), x[0].contiguous()), "shift must have shape"),
                       (lambda: moss.op_swiglu_i8(x), "must be torch.bfloat16"),
                       (lambda: moss.op_gemm_i8(i8, s[:3], i8, s), "a_scale must have shape"),
                       (lambda: moss.op_gemm_i8(i8, s, i8[:, :32].contiguous(), s), "must be \\[M, K\\]"),
                       (lambda: moss.op_gemm_i8(i8, s, i8, s, gate=s), "go together"),
                       (lambda: moss.op_gemm_i8(i8, s, i8, s, out=x), "out must have shape"),
                       (lambda: moss.op_gemm_i8(i8, s, i8, s, gate=s, residual=x[:, :4].contiguous(),
                                                out_dtype=torch.bfloat16), "writes FP32"),
                       (lambda: moss.op_qk_norm_rope(x.view(4, 1, 64), x.view(4, 1, 64).bfloat16(), None, None, None),
                        "q's tokens"),
                       (lambda: moss.op_qk_norm_rope(x.view(4, 1, 64), None, s, None, None), "q_gain must have shape"),
                       (lambda: moss.op_qk_norm_rope(x.view(4, 2, 32), None, None, None, None), "head_dim must be"),
                       (lambda: moss.op_qk_norm_rope(x.view(4, 1, 64), None, None, None, None, pairing="odd"), "pairing")):
        with pytest.raises(moss.MossError, match=what):
            call()


def test_empty_calls():
    e = torch.empty(0, 64, device="cuda")
    before = moss.launch_count()
    q, s = moss.op_quantize_i8(e)
    assert q.shape == (0, 64) and s.shape == (0,)
    assert moss.op_ln_modulate_i8(e, torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda"))[0].shape == (0, 64)
    assert moss.op_swiglu_i8(e.bfloat16())[0].shape == (0, 32)
    b, sb = ints(500, 7, 64), torch.ones(7, device="cuda")
    assert moss.op_gemm_i8(q, s, b, sb).shape == (0, 7)
    assert moss.op_qk_norm_rope(e.view(0, 1, 64), None, None, None, None)[0].shape == (0, 1, 64)
    assert moss.launch_count() == before
