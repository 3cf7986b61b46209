"""Host-side checks of the operators around the product (no GPU needed): what
the C ABI refuses before any HIP call, the size helpers, and what the binding
refuses before it reaches the library."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def bl():
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


P = 0x10000  # a fake, 16-byte aligned address: never dereferenced on these paths
import ctypes  # noqa: E402

ROWS = (ctypes.c_int64 * 9)(5, 3, 1, 1, 1, 1, 1, 1, 1)


def call(fn, order, defaults, kw):
    a = dict(defaults)
    unknown = set(kw) - set(a)
    assert not unknown, unknown
    a.update(kw)
    return fn(*[a[k] for k in order])


FWD = dict(xq=P, scale=P, packed=P, layout=0, gammas=P, rows=ROWS, nseg=2, M=32, K=64, bias=P, bdt=0, act=4,
           residual=P, rs=1.0, z=P, y=P, ydt=0, stream=None)
LIN = dict(x=P, xdt=1, packed=P, layout=0, gammas=P, rows=ROWS, nseg=2, M=2, K=64, bias=P, bdt=0, act=4, residual=P,
           rs=1.0, z=P, y=P, ydt=0, stream=None)
EBW = dict(gy=P, gydt=0, z=P, zdt=0, act=4, rs=1.0, M=8, N=40, gz=P, gzdt=0, gb=P, gr=P, ws=P, wsb=1 << 20,
           stream=None)
NRM = dict(h=P, hdt=0, block=P, xdt=1, rs=1.0, gate=P, gk=1, qk=1, qw=P, qb=P, qe=1e-5, pk=2, pw=P, pb=P, pe=1e-5,
           pdt=0, M=4, K=64, ho=P, n=P, xq=P, scale=P, stats=P, stream=None)
NBW = dict(G=P, gn=P, gndt=0, ho=P, hdt=0, block=P, xdt=1, stats=P, rs=1.0, gate=P, gk=1, qk=1, qw=P, qb=P, pk=2,
           pw=P, pdt=0, M=4, K=64, gh=P, gblk=P, ggate=P, gqw=P, gqb=P, gpw=P, gpb=P, ws=P, wsb=1 << 24, stream=None)


def fwd(bl, **kw):
    return call(bl.library().bitlinear_forward_epilogue, FWD, FWD, kw)


def lin(bl, **kw):
    return call(bl.library().bitlinear_linear_epilogue, LIN, LIN, kw)


def ebw(bl, **kw):
    return call(bl.library().bitlinear_epilogue_backward, EBW, EBW, kw)


def nrm(bl, **kw):
    return call(bl.library().bitlinear_block_norm, NRM, NRM, kw)


def nbw(bl, **kw):
    return call(bl.library().bitlinear_block_norm_backward, NBW, NBW, kw)


PRODUCT_BAD = [
    dict(packed=None), dict(gammas=None), dict(y=None), dict(packed=P + 8), dict(gammas=P + 2), dict(y=P + 4),
    dict(bias=P + 4), dict(residual=P + 8), dict(z=P + 2), dict(rows=None), dict(nseg=0), dict(nseg=9),
    dict(M=-1), dict(K=0), dict(K=16909321), dict(layout=3), dict(layout=-1), dict(ydt=2), dict(bdt=2), dict(bdt=-1),
    dict(act=-1), dict(act=6), dict(rs=math.inf), dict(rs=math.nan),
    dict(rows=(ctypes.c_int64 * 2)(4, 0)), dict(rows=(ctypes.c_int64 * 2)(2147483647, 1))]


@pytest.mark.parametrize("kw", PRODUCT_BAD + [dict(xq=None), dict(scale=None), dict(xq=P + 1), dict(M=65535 * 128 + 1)])
def test_forward_epilogue_rejects(bl, kw):
    assert fwd(bl, **kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", PRODUCT_BAD + [dict(x=None), dict(x=P + 2), dict(xdt=5)])
def test_linear_epilogue_rejects(bl, kw):
    assert lin(bl, **kw) == bl.BL_ERR_INVALID_ARG


def test_linear_epilogue_takes_at_most_four_tokens(bl):
    assert lin(bl, M=5) == bl.BL_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(gy=None), dict(z=None), dict(gy=P + 4), dict(z=P + 8), dict(gz=P + 2), dict(gb=P + 4), dict(gr=P + 4),
    dict(ws=P + 4), dict(ws=None), dict(wsb=0), dict(M=-1), dict(N=-1), dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 1),
    dict(gydt=2), dict(zdt=-1), dict(gzdt=9), dict(act=6), dict(act=-1), dict(rs=math.nan),
    dict(gz=None, gb=None, gr=None)])
def test_epilogue_backward_rejects(bl, kw):
    assert ebw(bl, **kw) == bl.BL_ERR_INVALID_ARG


def test_epilogue_backward_workspace_is_what_it_asks_for(bl):
    need = bl.bitlinear_epilogue_backward_workspace_bytes(8, 40)
    assert need > 0 and ebw(bl, wsb=need - 1) == bl.BL_ERR_INVALID_ARG
    # no bias gradient: no workspace
    for kw in (dict(wsb=need), dict(gb=None, ws=None, wsb=0), dict(act=0, z=None)):
        assert ebw(bl, **kw) in (bl.BL_ERR_DEVICE, bl.BL_OK) if not torch.cuda.is_available() else True
    for M, N in ((0, 5), (5, 0), (-1, 5), ((1 << 24) + 1, 5), (5, (1 << 24) + 1)):
        assert bl.bitlinear_epilogue_backward_workspace_bytes(M, N) == 0


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(ho=None), dict(h=P + 4), dict(block=P + 8), dict(gate=P + 4), dict(ho=P + 4), dict(n=P + 2),
    dict(xq=P + 4), dict(scale=P + 4), dict(stats=P + 4), dict(qw=P + 4), dict(qb=P + 4), dict(pw=P + 4),
    dict(pb=P + 4), dict(hdt=2), dict(xdt=2), dict(pdt=2), dict(gk=3), dict(gk=-1), dict(gk=0), dict(gate=None),
    dict(qk=3), dict(pk=-1), dict(qe=0.0), dict(qe=-1.0), dict(qe=math.nan), dict(pe=math.inf), dict(pe=0.0),
    dict(rs=math.inf), dict(rs=math.nan), dict(M=-1), dict(K=0), dict(K=16909321), dict(M=2147483648),
    dict(n=None, xq=None, scale=None), dict(xq=None), dict(scale=None),
    dict(qk=0), dict(pk=0),                                # parameters without their norm
    dict(pk=0, pw=None, pb=None),                          # n without norm_pre
    dict(block=None), dict(block=None, ho=None),           # a gate or norm_post without a block
    dict(block=None, ho=None, gate=None, gk=0),
    dict(block=None, gate=None, gk=0, qk=0, qw=None, qb=None),   # h_out without a block
    dict(block=None, ho=None, gate=None, gk=0, qk=0, qw=None, qb=None, pk=0, pw=None, pb=None, n=None, xq=None,
         scale=None)])
def test_block_norm_rejects(bl, kw):
    assert nrm(bl, **kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(gn=None), dict(ho=None), dict(stats=None), dict(gh=None), dict(ws=None), dict(wsb=64), dict(G=P + 4),
    dict(gn=P + 4), dict(ho=P + 4), dict(block=P + 4), dict(stats=P + 4), dict(gate=P + 4), dict(gh=P + 4),
    dict(gblk=P + 4), dict(ggate=P + 4), dict(gqw=P + 4), dict(gqb=P + 4), dict(gpw=P + 4), dict(gpb=P + 4),
    dict(ws=P + 4), dict(hdt=2), dict(xdt=-1), dict(gndt=2), dict(pdt=7), dict(gk=3), dict(gk=0), dict(gate=None),
    dict(qk=3), dict(pk=3), dict(rs=math.nan), dict(M=-1), dict(K=0), dict(K=(1 << 24) + 1), dict(M=(1 << 24) + 1),
    dict(qk=0, qw=None, qb=None),                          # norm_post's gradients without it
    dict(pk=0, pw=None, gn=None),                          # norm_pre's
    dict(pk=0, pw=None, gpw=None, gpb=None),               # grad_n without norm_pre
    dict(block=None), dict(block=None, gblk=None),
    dict(block=None, gblk=None, gate=None, gk=0, ggate=None)])
def test_block_norm_backward_rejects(bl, kw):
    assert nbw(bl, **kw) == bl.BL_ERR_INVALID_ARG


def test_block_norm_backward_workspace(bl):
    need = bl.bitlinear_block_norm_backward_workspace_bytes(4, 64)
    assert need > 0 and nbw(bl, wsb=need - 1) == bl.BL_ERR_INVALID_ARG
    for M, K in ((0, 64), (4, 0), ((1 << 24) + 1, 4), (4, (1 << 24) + 1)):
        assert bl.bitlinear_block_norm_backward_workspace_bytes(M, K) == 0


def test_empty_batches_are_noops(bl):
    assert fwd(bl, M=0) == bl.BL_OK and lin(bl, M=0) == bl.BL_OK and nrm(bl, M=0) == bl.BL_OK
    assert fwd(bl, M=0, xq=None, y=None, z=None) == bl.BL_OK
    assert ebw(bl, N=0) == bl.BL_OK
    assert ebw(bl, M=0, gy=None, z=None, gb=None) == bl.BL_OK
    assert nbw(bl, M=0, ggate=None, gqw=None, gqb=None, gpw=None, gpb=None) == bl.BL_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")
def test_valid_calls_stop_at_the_device_check(bl):
    for f in (fwd, lin, ebw, nrm, nbw):
        assert f(bl) == bl.BL_ERR_DEVICE, f


# ---- the binding ---------------------------------------------------------------
def tensors():
    return dict(xq=torch.zeros(5, 64, dtype=torch.int8), scale=torch.ones(5), packed=torch.zeros(8, 16, dtype=torch.uint8),
                gammas=torch.ones(1), seg_rows=8, K=64)


@pytest.mark.parametrize("kw,word", [
    (dict(xq=torch.zeros(5, 64)), "xq"), (dict(xq=torch.zeros(64, dtype=torch.int8)), "xq"), (dict(K=65), "xq"),
    (dict(scale=torch.ones(4)), "scale"), (dict(packed=torch.zeros(8, 32, dtype=torch.uint8)), "packed"),
    (dict(packed=torch.zeros(9, 16, dtype=torch.uint8)), "packed"), (dict(gammas=torch.ones(1, dtype=torch.float64)), "gammas"),
    (dict(seg_rows=(4, 4)), "gammas"), (dict(bias=torch.ones(7)), "bias"), (dict(bias=torch.ones(8, dtype=torch.float16)), "bias"),
    (dict(act="tanh"), "act"), (dict(layout="3bit"), "layout"), (dict(residual=torch.ones(8, 5).t(), y=torch.ones(5, 8)), "contiguous"),
    (dict(residual=torch.ones(5, 8), y=torch.ones(5, 8, dtype=torch.bfloat16)), "residual"),
    (dict(residual=torch.ones(5, 8, dtype=torch.float16)), "out_dtype"), (dict(y=torch.ones(4, 8)), "y"),
    (dict(z=torch.ones(5, 9)), "z"), (dict(residual_scale=float("nan")), "residual_scale"),
    (dict(out_dtype=torch.float64), "out_dtype"), ({}, "cpu")])
def test_binding_refuses_product_arguments(bl, kw, word):
    with pytest.raises(bl.BitLinearError, match=word) as e:
        bl.bitlinear_forward_epilogue(**{**tensors(), **kw})
    assert e.value.status == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,word", [
    (dict(h=torch.ones(64)), "h is"), (dict(h=torch.ones(5, 64, dtype=torch.float16)), "h is"),
    (dict(block=torch.ones(5, 63)), "block"), (dict(gate=torch.ones(63)), "gate"),
    (dict(gate=torch.ones(5, 64, dtype=torch.bfloat16)), "gate"), (dict(gate=torch.ones(64, dtype=torch.bfloat16)), "gate"),
    (dict(h_out=torch.ones(5, 64, dtype=torch.bfloat16)), "h_out"), (dict(n=torch.ones(5, 64, dtype=torch.bfloat16)), "n is"),
    (dict(out_dtype=torch.bfloat16), "out_dtype"), (dict(stats=torch.ones(5, 3)), "stats"),
    (dict(pre=None, n=torch.ones(5, 64)), "norm"), (dict(residual_scale=float("inf")), "residual_scale"),
    (dict(h=torch.ones(64, 5).t()), "contiguous"), ({}, "cpu")])
def test_binding_refuses_norm_arguments(bl, kw, word):
    a = dict(h=torch.ones(5, 64), block=torch.ones(5, 64), pre=bl.Norm("rms", torch.ones(64)),
             post=bl.Norm("layer", torch.ones(64), torch.ones(64)), gate=torch.ones(64))
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_block_norm(**{**a, **kw})


def test_binding_refuses_mixed_parameter_types(bl):
    with pytest.raises(bl.BitLinearError, match="pre.weight"):
        bl.bitlinear_block_norm(torch.ones(5, 64), torch.ones(5, 64), pre=bl.Norm("rms", torch.ones(64, dtype=torch.bfloat16)),
                                post=bl.Norm("rms", torch.ones(64)))
    with pytest.raises(bl.BitLinearError, match="kind"):
        bl.bitlinear_block_norm(torch.ones(5, 64), pre=bl.Norm("batch", torch.ones(64)))


@pytest.mark.parametrize("kw,word", [
    (dict(grad_n=torch.ones(5, 63)), "grad_n"), (dict(stats=torch.ones(4, 4)), "stats"),
    (dict(grad_h_out=torch.ones(5, 64, dtype=torch.bfloat16)), "grad_h_out"), (dict(grad_gate=torch.ones(5, 64)), "grad_gate"),
    (dict(grad_pre_weight=torch.ones(64, dtype=torch.bfloat16)), "grad_pre_weight"), ({}, "cpu")])
def test_binding_refuses_norm_backward_arguments(bl, kw, word):
    a = dict(grad_h_out=torch.ones(5, 64), grad_n=torch.ones(5, 64), h_out=torch.ones(5, 64), block=torch.ones(5, 64),
             stats=torch.ones(5, 4), pre=bl.Norm("rms", torch.ones(64)), gate=torch.ones(64))
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_block_norm_backward(**{**a, **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(grad_y=torch.ones(5)), "grad_y"), (dict(z=torch.ones(5, 9)), "z has"), (dict(act="swish"), "act"),
    (dict(grad_bias=torch.ones(9)), "grad_bias"), (dict(grad_residual=torch.ones(5, 8, dtype=torch.bfloat16)), "grad_residual"),
    (dict(out_dtype=torch.float16), "out_dtype"), ({}, "cpu")])
def test_binding_refuses_epilogue_backward_arguments(bl, kw, word):
    a = dict(grad_y=torch.ones(5, 8), z=torch.ones(5, 8), act="gelu")
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_epilogue_backward(**{**a, **kw})


def test_binding_refuses_a_stream_of_another_device(bl):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    st, t, h = Stream(), tensors(), torch.ones(5, 64)
    w = (t["packed"], t["gammas"], 8)
    for f in (lambda: bl.bitlinear_forward_epilogue(**t, stream=st), lambda: bl.bitlinear_linear_epilogue(h[:2], *w, stream=st),
              lambda: bl.linear_epilogue(h, *w, stream=st), lambda: bl.bitlinear_epilogue_backward(h, h, "silu", stream=st),
              lambda: bl.bitlinear_block_norm(h, pre=bl.Norm(), stream=st),
              lambda: bl.bitlinear_block_norm_backward(None, h, h, None, torch.ones(5, 4), pre=bl.Norm(), stream=st)):
        with pytest.raises(bl.BitLinearError, match="stream is of cuda:1"):
            f()


@pytest.mark.parametrize("shape", [(), (64,), (1, 5, 64)])
def test_binding_refuses_activations_of_other_ranks(bl, shape):
    t = tensors()
    for f in (bl.linear_epilogue, bl.bitlinear_linear_epilogue):
        with pytest.raises(bl.BitLinearError, match="x is"):
            f(torch.ones(shape), t["packed"], t["gammas"], 8)


def test_segment_rows_are_read_at_each_call(bl):
    """Row counts held in 0-d tensors are taken as the numbers they are at the call:
    a changed count is a changed stack (refused here for its packed rows)."""
    rows = [torch.tensor(4), torch.tensor(4)]
    args = {**tensors(), "gammas": torch.ones(2), "seg_rows": rows}
    for more, word in ((0, "cpu"), (1, "packed")):
        rows[0] += more
        with pytest.raises(bl.BitLinearError, match=word):
            bl.bitlinear_forward_epilogue(**args)
        with pytest.raises(bl.BitLinearError, match=word):
            bl.bitlinear_linear_epilogue(torch.ones(2, 64), args["packed"], args["gammas"], tuple(rows))


def test_row_bytes_are_those_of_the_call(bl):
    """K held in a 0-d tensor is the number that it is at the call: packed rows of
    another K are refused."""
    K = torch.tensor(64)
    for k, word in ((64, "cpu"), (128, "packed")):
        K.fill_(k)
        with pytest.raises(bl.BitLinearError, match=word):
            bl.bitlinear_forward_epilogue(**{**tensors(), "xq": torch.zeros(5, k, dtype=torch.int8), "K": K})
