"""The 8-bit linear path where its arithmetic, its sizes and its streams come to their ends, against 64 bits."""
import time

import pytest
import torch

import diffusion_transformer_text_block_b200 as moss
from tests.test_gpu_i8 import check_gemm, check_rows_of, gemm_case, no_device_error, randn, swiglu_reference  # noqa: F401 (a fixture among them)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ rows to 8 bits
GATES = [-86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -93.0, -104.0, -120.0, -150.0, -174.0]


@pytest.mark.parametrize("dim", [16, 1024, 8192])
def test_swiglu_gates_far_below_zero(dim):
    """Rows of one gate each, for which e^-g leaves FP32's range, times u from 1e37 to 3e38: SiLU(g) u is a number.
    __expf(g/2) twice is within 2 (2 + 1.173 |g| / 2) ulp (2 u each), the three products add 3 u: below the
    reference's bound; 2^-140 is far above what a subnormal intermediate could add and far below every h."""
    gu = torch.empty(len(GATES), 2 * dim, device="cuda", dtype=torch.bfloat16)
    gu[:, :dim] = torch.tensor(GATES, device="cuda")[:, None]
    gu[:, dim:] = (1e37 * 30 ** torch.rand(len(GATES), dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
                   * torch.sign(randn(2, len(GATES), dim))).bfloat16()
    q, scale = moss.op_swiglu_i8(gu)
    h, err = swiglu_reference(gu)
    assert (h.abs().amax(dim=1) > 2.0 ** -126).all()
    check_rows_of(q, scale, h, err + 2.0 ** -140)
    assert (q.abs().amax(dim=1) == 127).all()


def test_swiglu_far_gates_beside_others():
    """A far gate changes none of its neighbours, and gives a tiny value or 0 beside them as it should."""
    gu = randn(3, 6, 2 * 704, scale=2.0).bfloat16()
    gu[:, 5] = 0
    want = moss.op_swiglu_i8(gu)
    gu[:, 5], gu[:, 704 + 5] = -88.0, 1.0
    q, scale = moss.op_swiglu_i8(gu)
    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])
    gu[0, 9], gu[0, 704 + 9] = float("-inf"), 1.0
    gu[1, 9], gu[1, 704 + 9] = -200.0, float("inf")
    gu[2, 9], gu[2, 704 + 9] = -1e30, 3e38
    q, scale = moss.op_swiglu_i8(gu)
    assert torch.isnan(scale[:2]).all() and (q[:2] == 0).all()
    assert torch.isfinite(scale[2:]).all() and q[2, 9] == 0


# ------------------------------------------------------------------------------ streams
def every_operator():
    """name: a call of it with nothing but stream= to fill in; the outputs of each are larger than a megabyte."""
    x, mod = randn(10, 512, 4096), randn(11, 4096, scale=0.1)
    gu = randn(12, 512, 8192).bfloat16()
    a, b = moss.op_quantize_i8(x), moss.op_quantize_i8(randn(13, 4096, 4096))
    heads, rope = randn(14, 512, 32, 128).bfloat16(), moss.op_rope_table(16, 32, 0)
    return {"quantize": lambda s: moss.op_quantize_i8(x, stream=s),
            "ln_modulate": lambda s: moss.op_ln_modulate_i8(x, mod, mod, stream=s),
            "swiglu": lambda s: moss.op_swiglu_i8(gu, stream=s),
            "gemm": lambda s: (moss.op_gemm_i8(*a, *b, stream=s),),
            "qk_norm_rope": lambda s: moss.op_qk_norm_rope(heads, heads, None, None, rope, stream=s),
            "rope_table": lambda s: (moss.op_rope_table(64, 64, 512, stream=s),)}


OPERATORS = ["quantize", "ln_modulate", "swiglu", "gemm", "qk_norm_rope", "rope_table"]


@pytest.mark.parametrize("name", OPERATORS)
@pytest.mark.parametrize("by_handle", [False, True])
def test_new_tensors_come_from_the_given_streams_pool(name, by_handle):
    """Blocks of the outputs' sizes lie free in the current stream's pool: work of that stream which is still under
    way may use them, so a call on another stream must not take them."""
    call = every_operator()[name]
    want = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    spare = [torch.empty_like(w) for w in want for _ in range(3)]
    free = {t.data_ptr() for t in spare if t.numel() * t.element_size() > 1 << 20}
    assert free
    del spare
    got = call(s.cuda_stream if by_handle else s)
    torch.cuda.synchronize()
    assert not free & {g.data_ptr() for g in got}
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("name", OPERATORS)
def test_a_call_on_a_given_stream_does_not_wait_for_the_current_one(name):
    """The current stream is busy for some tenths of a second; the call's stream is done long before."""
    call = every_operator()[name]
    s = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    call(s)  # the stream's pool has its blocks: no allocation below waits for the device
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(600_000_000)
    busy.record()
    got = call(s)
    s.synchronize()
    done = busy.query()
    torch.cuda.synchronize()
    assert not done
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_rope_table_sizes():
    for args in ((1 << 32, 0, 3), (4, 4, 1 << 32), (1 << 12, 1 << 12, 1), (5000, 5000, 0)):
        with pytest.raises(moss.MossError):
            moss.op_rope_table(*args)


# ------------------------------------------------------------------------------ waits that give up
@pytest.mark.parametrize("failure,M,N,K", [("lost load", 77, 704, 1024), ("lost load", 300, 300, 256),
                                           ("lost load, pair", 3840, 3840, 1280), ("kept accumulator", 3840, 3840, 1280),
                                           ("kept accumulator", 3840, 3840, 256)])
def test_gemm_wait_gives_up_and_every_warp_finishes(failure, M, N, K):
    """A load that never comes, or an accumulator that is never handed back: the bounded waits give up (2 s, some
    of them behind others), the launch ends, and the next launches compute as before."""
    a, sa, b, sb, *_ = gemm_case(80, M, N, K, False, False)
    want = moss.op_gemm_i8(a, sa, b, sb)
    assert moss.device_status(clear=True) == 0
    t0 = time.time()
    moss.selftest_gemm_i8_timeout(failure, a, sa, b, sb)
    status = moss.device_status(clear=True)  # synchronises
    assert status in (0x111, 0x112, 0x113)
    assert 1.0 < time.time() - t0 < 60.0
    for _ in range(2):
        assert torch.equal(moss.op_gemm_i8(a, sa, b, sb), want)
        assert moss.device_status(clear=True) == 0


# ------------------------------------------------------------------------------ sizes
@pytest.mark.parametrize("tokens", [True, False])
def test_gemm_of_the_largest_size(tokens):
    """2^31 - 1 tokens by one channel, and one token by as many channels (47 GB each): every output right."""
    big = 2 ** 31 - 1
    wide = torch.ones(big, 16, device="cuda", dtype=torch.int8)
    scale = torch.ones(big, device="cuda")
    one, unit = torch.ones(1, 16, device="cuda", dtype=torch.int8), torch.ones(1, device="cuda")
    at = torch.tensor([0, 1, 255, 256, 2 ** 30 + 77, big - 258, big - 257, big - 256, big - 255, big - 2, big - 1], device="cuda")
    wide[at] = torch.randint(-127, 128, (len(at), 16), generator=torch.Generator("cuda").manual_seed(90), device="cuda",
                             dtype=torch.int8)
    scale[at] = 0.5 + torch.arange(len(at), device="cuda")
    c = moss.op_gemm_i8(wide, scale, one, unit) if tokens else moss.op_gemm_i8(one, unit, wide, scale)
    c = c.view(-1)
    check_gemm(c[at][:, None], wide[at], scale[at], one, unit, None, None, None)
    c[at] = 16.0
    right = bool((c == 16).all())
    del c, wide, scale
    torch.cuda.empty_cache()
    assert right


@pytest.mark.parametrize("M,N,K,form", [(9216, 9216, 3072, "bf16"), (4429, 3072, 8192, "resid"), (9216, 3072, 3072, "f32"),
                                        (5001, 4100, 2688, "bias"), (2304, 9216, 912, "resid")])
def test_gemm_of_many_tiles_a_pair(M, N, K, form):
    """Three tiles and more for a CTA pair, each of many K slots (24, 64, 24, 21 and 8 of a ring of 7): both
    accumulators and every slot are used again and again.  Every output against 64 bits."""
    args = gemm_case(95, M, N, K, form in ("bias", "resid"), form == "resid")
    a, sa, b, sb, bias, gate, res = args
    c = moss.op_gemm_i8(a, sa, b, sb, bias=bias, gate=gate, residual=res,
                        out_dtype=torch.float32 if form in ("f32", "resid") else torch.bfloat16)
    assert -(-M // 256) * -(-N // 256) > 2 * 74
    for r in range(0, M, 1024):
        rows = slice(r, r + 1024)
        check_gemm(c[rows], a[rows], sa[rows], b, sb, bias, gate, res[rows] if res is not None else None)
