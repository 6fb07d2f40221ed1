"""Argument checks of the 8-bit linear path and of the query/key norm with rotation, without a GPU:
a refused call launches nothing, and an empty one does nothing."""
import ctypes

import pytest
import torch

import diffusion_transformer_text_block_b200 as moss

INVALID, ABI, UNSUPPORTED = 1, 5, 6
P = ctypes.c_void_p
BASE = 1 << 20  # addresses that nothing reads: every call below is refused before a launch


def at(k):
    """A made-up 16-byte aligned address, 1 MB from its neighbours."""
    return P(BASE * (k + 1))


@pytest.fixture(autouse=True)
def nothing_launched():
    before = moss.launch_count()
    yield
    assert moss.launch_count() == before


def said():
    return moss.lib().moss_last_error().decode()


def test_quantize_refusals():
    f = moss.lib().moss_op_quantize_i8

    def call(x=at(0), dt=moss.DTYPE_BF16, stride=64, q=at(1), s=at(2), rows=4, dim=64):
        return f(x, dt, stride, q, s, rows, dim, None)

    for kw in (dict(dt=2), dict(dt=-1), dict(rows=-1), dict(dim=0), dict(dim=8), dict(dim=24), dict(dim=32784, stride=32784),
               dict(stride=63), dict(stride=68), dict(stride=66, dt=moss.DTYPE_F32), dict(stride=(1 << 46) + 8), dict(stride=1 << 30, rows=1 << 20),
               dict(x=None), dict(q=None), dict(s=None), dict(x=P(BASE + 8)), dict(q=P(BASE * 2 + 8)), dict(s=P(BASE * 3 + 2)),
               dict(q=at(0)), dict(s=at(0)), dict(s=at(1)), dict(q=P(BASE + 3 * 128 + 112))):
        assert call(**kw) == INVALID, kw
        assert said(), kw
    assert call(x=None, q=None, s=None, rows=0) == 0


def test_ln_modulate_refusals():
    f = moss.lib().moss_op_ln_modulate_i8

    def call(x=at(0), sh=at(1), sc=at(2), q=at(3), s=at(4), rows=4, dim=64):
        return f(x, sh, sc, q, s, rows, dim, None)

    for kw in (dict(rows=-1), dict(dim=0), dict(dim=72), dict(dim=65536), dict(x=None), dict(sh=None), dict(sc=None),
               dict(q=None), dict(s=None), dict(x=P(BASE + 4)), dict(sh=P(BASE * 2 + 8)), dict(q=at(0)), dict(q=at(1)),
               dict(s=at(2)), dict(s=at(3))):
        assert call(**kw) == INVALID, kw
    assert call(x=None, sh=None, sc=None, q=None, s=None, rows=0) == 0


def test_swiglu_refusals():
    f = moss.lib().moss_op_swiglu_i8

    def call(gu=at(0), stride=128, q=at(1), s=at(2), rows=4, dim=64):
        return f(gu, stride, q, s, rows, dim, None)

    for kw in (dict(rows=-1), dict(dim=0), dict(dim=40), dict(stride=127), dict(stride=132), dict(gu=None), dict(q=None),
               dict(s=None), dict(gu=P(BASE + 2)), dict(q=at(0)), dict(s=at(1))):
        assert call(**kw) == INVALID, kw
    assert call(gu=None, q=None, s=None, rows=0) == 0


def test_gemm_refusals():
    f = moss.lib().moss_op_gemm_i8

    def call(a=at(0), sa=at(1), b=at(2), sb=at(3), bias=None, gate=None, resid=None, c=at(4), dt=moss.DTYPE_BF16, M=4,
             N=32, K=64):
        return f(a, sa, b, sb, bias, gate, resid, c, dt, M, N, K, None)

    f32 = moss.DTYPE_F32
    for kw in (dict(dt=3), dict(M=-1), dict(N=0), dict(K=0), dict(K=8), dict(K=72), dict(K=65552), dict(a=None), dict(sa=None),
               dict(b=None), dict(sb=None), dict(c=None), dict(a=P(BASE + 8)), dict(b=P(BASE * 3 + 1)), dict(c=P(BASE * 5 + 2)),
               dict(sa=P(BASE * 2 + 2)), dict(bias=P(BASE * 6 + 1)), dict(gate=at(5)), dict(resid=at(5), dt=f32),
               dict(gate=at(5), resid=at(6)), dict(gate=at(5), resid=P(BASE * 7 + 4), dt=f32), dict(c=at(0)), dict(c=at(1)),
               dict(c=at(2)), dict(c=at(3)), dict(bias=at(4)), dict(gate=at(4), resid=at(6), dt=f32),
               dict(gate=at(5), resid=P(BASE * 5 + 16), dt=f32), dict(M=1 << 30, N=1 << 20), dict(M=(1 << 31) - 1, N=(1 << 31) - 1)):
        assert call(**kw) == INVALID, kw
    assert call(a=None, sa=None, b=None, sb=None, c=None, M=0) == 0


def qk_args(**kw):
    a = moss.QkNormRopeArgs()
    moss.lib().moss_qk_norm_rope_args_init(ctypes.byref(a), ctypes.sizeof(moss.QkNormRopeArgs))
    a.rows, a.heads_q, a.heads_k, a.n_pos = 4, 2, 2, 16
    a.q_stride = a.k_stride = a.q_out_stride = a.k_out_stride = 256
    a.q, a.k, a.q_out, a.k_out, a.rope = (BASE * i for i in (1, 2, 3, 4, 5))
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def qk(**kw):
    return moss.lib().moss_op_qk_norm_rope(ctypes.byref(qk_args(**kw)), None)


def test_qk_defaults():
    a = moss.QkNormRopeArgs()
    moss.lib().moss_qk_norm_rope_args_init(ctypes.byref(a), ctypes.sizeof(moss.QkNormRopeArgs))
    assert a.struct_size == ctypes.sizeof(moss.QkNormRopeArgs)
    assert (a.in_dtype, a.out_dtype, a.head_dim, a.rot_dim, a.pairing) == (1, 1, 128, 128, 0)
    assert abs(a.eps - 1e-6) < 1e-12 and not a.q and not a.rope and a.rows == 0


def test_qk_refusals():
    assert moss.lib().moss_op_qk_norm_rope(None, None) == INVALID
    assert qk(struct_size=16) == ABI
    assert qk(head_dim=96) == UNSUPPORTED
    for kw in (dict(in_dtype=2), dict(out_dtype=-1), dict(pairing=2), dict(rot_dim=-8), dict(rot_dim=136), dict(rot_dim=12),
               dict(rows=-1), dict(heads_q=0), dict(heads_k=-1), dict(heads_q=70000), dict(eps=-1.0), dict(eps=float("nan")), dict(reserved=1),
               dict(q_stride=255), dict(k_stride=248), dict(q_out_stride=260), dict(k_out_stride=0),
               dict(q_stride=(1 << 46) + 8), dict(k_out_stride=1 << 30, rows=1 << 20), dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(rope=None),
               dict(n_pos=0), dict(rot_dim=0, positions=BASE * 9), dict(q=BASE + 8), dict(k_out=BASE * 4 + 2),
               dict(q_gain=BASE * 8 + 4), dict(positions=BASE * 9 + 2), dict(rope=BASE * 5 + 8),
               dict(q_out=BASE + 16), dict(k_out=BASE * 2 + 512),                                # shifted onto their input
               dict(q_out=BASE, q_out_stride=264),                                               # in place, other stride
               dict(q_out=BASE, out_dtype=0, k_out=BASE * 2),                                    # in place, other type
               dict(q_out=BASE * 2, q_out_stride=256), dict(k_out=BASE), dict(k_out=BASE * 3),   # another's buffer
               dict(q_out=BASE * 5), dict(q_gain=BASE * 3), dict(positions=BASE * 4)):           # an output over an operand
        assert qk(**kw) == INVALID, kw
        assert said(), kw
    assert qk(rows=0, q=None, k=None, q_out=None, k_out=None, rope=None) == 0


def test_qk_fused_buffer_columns_do_not_overlap():
    """q and k side by side in one buffer, in place: refused only for the missing table, that is after
    the overlap rules have been passed by a table-less twin."""
    w = 3 * 256
    fused = dict(q=BASE, k=BASE + 512, q_out=BASE, k_out=BASE + 512, q_stride=w, k_stride=w, q_out_stride=w, k_out_stride=w)
    assert qk(**fused, rope=BASE + 1024) == INVALID and "angles" in said()      # the table inside the buffer
    assert qk(**dict(fused, k_out=BASE + 256)) == INVALID and "overlap" in said()


def test_rope_table_refusals():
    f = moss.lib().moss_op_rope_table
    for args in ((at(0), -1, 4, 0), (at(0), 4, -1, 0), (at(0), 4, 4, -1), (at(0), 1 << 13, 1 << 12, 0), (None, 4, 4, 0),
                 (P(BASE + 8), 4, 4, 0)):
        assert f(*args, None) == INVALID, args
    assert f(None, 0, 7, 0, None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: moss.op_quantize_i8(x), lambda: moss.op_ln_modulate_i8(x, x[0], x[0]),
                 lambda: moss.op_swiglu_i8(x.bfloat16()),
                 lambda: moss.op_gemm_i8(x.char(), x[:, 0], x.char(), x[:, 0]),
                 lambda: moss.op_qk_norm_rope(x.view(4, 1, 64), None, None, None, None)):
        with pytest.raises(moss.MossError, match="must be a CUDA tensor"):
            call()


def test_the_packed_arguments_are_the_structure():
    """The binding packs the query/key arguments in one go: field for field what the structure declares."""
    n = len(moss.QkNormRopeArgs._fields_)
    values = [float(i) if name == "eps" else i + 1 for i, (name, _) in enumerate(moss.QkNormRopeArgs._fields_)]
    a = moss.QkNormRopeArgs.from_buffer_copy(moss._pack_qk(*values))
    assert [getattr(a, name) for name, _ in moss.QkNormRopeArgs._fields_] == values and n == 24
