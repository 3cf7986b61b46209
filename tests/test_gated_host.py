"""Host-side checks of the gated products, the 8-bit checkpoints and the gradients
from codes and stacks (no GPU needed): what the C ABI refuses before any HIP call,
the size helpers, and what the binding refuses before it reaches the library."""
import ctypes

import pytest
import torch

P = 0x10000  # a fake, 16-byte aligned address: never dereferenced on these paths
ROWS = (ctypes.c_int64 * 9)(5, 3, 1, 1, 1, 1, 1, 1, 1)
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def bl():
    from ternary_weight_linear_bitlinear_amd import bitlinear
    return bitlinear


FWD = dict(xq=P, scale=P, packed=P, layout=0, gammas=P, F=20, M=32, K=64, bias=P, bdt=0, act=3, z=P, codes=P, cs=P, y=P,
           ydt=0, stream=None)
LIN = dict(x=P, xdt=1, packed=P, layout=0, gammas=P, F=20, M=2, K=64, bias=P, bdt=0, act=3, z=P, y=P, ydt=0, stream=None)
BWD = dict(gy=P, gydt=0, z=P, zdt=0, codes=None, cs=None, act=3, M=200, F=20, gz=P, gzdt=0, gb=P, ws=P, wsb=1 << 20,
           stream=None)
KEEP = dict(x=P, xdt=0, M=8, K=70, codes=P, scale=P, stream=None)
BACK = dict(codes=P, scale=P, M=8, K=70, y=P, ydt=0, stream=None)
WGT = dict(gy=P, gydt=0, xq=P, scale=P, M=64, N=40, K=50, gw=P, gwdt=0, ws=P, wsb=1 << 40, stream=None)
INP = dict(gy=P, gydt=0, packed=P, layout=0, gammas=P, rows=ROWS, nseg=2, M=64, K=50, gx=P, gxdt=0, ws=P, wsb=1 << 40,
           stream=None)


def call(bl, name, defaults, kw):
    assert not set(kw) - set(defaults), kw
    return getattr(bl.library(), name)(*{**defaults, **kw}.values())


PRODUCT_BAD = [dict(packed=None), dict(gammas=None), dict(y=None), dict(packed=P + 8), dict(gammas=P + 2), dict(y=P + 4),
               dict(bias=P + 4), dict(z=P + 2), dict(F=0), dict(F=-1), dict(F=1 << 30), dict(F=1 << 40), dict(M=-1),
               dict(K=0), dict(K=16909321), dict(layout=3), dict(layout=-1), dict(ydt=2), dict(bdt=2), dict(bdt=-1),
               dict(act=-1), dict(act=6)]


@pytest.mark.parametrize("kw", PRODUCT_BAD + [
    dict(xq=None), dict(scale=None), dict(xq=P + 1), dict(scale=P + 4), dict(M=65535 * 128 + 1), dict(codes=None),
    dict(cs=None), dict(codes=P + 8), dict(cs=P + 4)])
def test_forward_rejects(bl, kw):
    assert call(bl, "bitlinear_forward_gated", FWD, kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", PRODUCT_BAD + [dict(x=None), dict(x=P + 2), dict(xdt=5)])
def test_linear_rejects(bl, kw):
    assert call(bl, "bitlinear_linear_gated", LIN, kw) == bl.BL_ERR_INVALID_ARG


def test_linear_takes_at_most_four_tokens(bl):
    assert call(bl, "bitlinear_linear_gated", LIN, dict(M=5)) == bl.BL_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(gy=None), dict(z=None), dict(codes=P), dict(cs=P), dict(codes=P, cs=P), dict(z=None, codes=P),
    dict(z=None, cs=P), dict(gy=P + 4), dict(z=P + 8), dict(z=None, codes=P + 8, cs=P), dict(z=None, codes=P, cs=P + 4),
    dict(gz=P + 2), dict(gb=P + 4), dict(ws=P + 4), dict(ws=None), dict(wsb=0), dict(M=-1), dict(F=-1),
    dict(M=(1 << 23) + 1), dict(F=(1 << 23) + 1), dict(gydt=2), dict(zdt=-1), dict(gzdt=9), dict(act=6), dict(act=-1),
    dict(gz=None, gb=None)])
def test_backward_rejects(bl, kw):
    assert call(bl, "bitlinear_gated_backward", BWD, kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(codes=None), dict(scale=None), dict(x=P + 4), dict(codes=P + 8),
                                dict(scale=P + 4), dict(xdt=2), dict(M=-1), dict(K=0), dict(M=(1 << 24) + 1),
                                dict(K=(1 << 24) + 1)])
def test_checkpoint_rejects(bl, kw):
    assert call(bl, "bitlinear_checkpoint", KEEP, kw) == bl.BL_ERR_INVALID_ARG
    kw = {{"x": "y", "xdt": "ydt"}.get(k, k): v for k, v in kw.items()}
    assert call(bl, "bitlinear_checkpoint_restore", BACK, kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(gy=None), dict(xq=None), dict(scale=None), dict(gw=None), dict(gy=P + 4), dict(xq=P + 8),
                                dict(scale=P + 4), dict(gw=P + 4), dict(ws=P + 4), dict(gydt=2), dict(gwdt=2), dict(M=-1),
                                dict(N=-1), dict(K=0), dict(M=(1 << 24) + 1), dict(N=(1 << 24) + 1), dict(K=(1 << 24) + 1),
                                dict(M=4096, N=1024, K=1024, ws=None), dict(M=4096, N=1024, K=1024, wsb=64)])
def test_weight_rejects(bl, kw):
    assert call(bl, "bitlinear_backward_weight_codes", WGT, kw) == bl.BL_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(gy=None), dict(packed=None), dict(gammas=None), dict(gx=None), dict(gy=P + 4),
                                dict(packed=P + 8), dict(gammas=P + 2), dict(gx=P + 4), dict(ws=P + 4), dict(gydt=2),
                                dict(gxdt=2), dict(layout=3), dict(rows=None), dict(nseg=0), dict(nseg=9), dict(M=-1),
                                dict(K=0), dict(M=(1 << 24) + 1), dict(K=(1 << 24) + 1),
                                dict(rows=(ctypes.c_int64 * 2)(1 << 23, 1)), dict(rows=(ctypes.c_int64 * 2)(4, 0)),
                                dict(rows=(ctypes.c_int64 * 2)(8192, 8192), M=512, K=4096, ws=None),
                                dict(rows=(ctypes.c_int64 * 2)(8192, 8192), M=512, K=4096, wsb=64)])
def test_input_rejects(bl, kw):
    assert call(bl, "bitlinear_backward_input_segmented", INP, kw) == bl.BL_ERR_INVALID_ARG


def test_sizes(bl):
    lib = bl.library()
    for K in (-5, 0, 1, 63, 64, 65, 4096, 11008, 1 << 24):
        assert lib.bitlinear_checkpoint_groups(K) == bl.bitlinear_checkpoint_groups(K) == max(0, -(-K // 64))
    for M, F in ((0, 5), (5, 0), (-1, 5), ((1 << 23) + 1, 5), (5, (1 << 23) + 1)):
        assert bl.bitlinear_gated_backward_workspace_bytes(M, F) == 0
    assert bl.bitlinear_gated_backward_workspace_bytes(128, 20) == 0  # one run of rows: no partial sums
    need = bl.bitlinear_gated_backward_workspace_bytes(200, 20)
    assert need > 0 and call(bl, "bitlinear_gated_backward", BWD, dict(wsb=need - 1)) == bl.BL_ERR_INVALID_ARG
    for M, N, K in ((0, 5, 5), (5, 0, 5), (5, 5, 0), ((1 << 24) + 1, 5, 5)):
        assert bl.bitlinear_backward_weight_codes_workspace_bytes(M, N, K) == 0
        assert bl.bitlinear_backward_input_segmented_workspace_bytes(M, N, K) == 0
    # partial sums of a few workgroups for each tile, never more than sixteen
    for a in ((4096, 256, 256), (4096, 4096, 4096), (200, 2003, 3000), (64, 8192, 4096), (1, 1, 1), (16, 1 << 23, 8)):
        for d in (torch.float32, BF16):
            w, x = (f(*a, d) for f in (bl.bitlinear_backward_weight_codes_workspace_bytes,
                                       bl.bitlinear_backward_input_segmented_workspace_bytes))
            assert 0 <= w <= 4 * (16 * a[1] * a[2] + 4 + 64 * a[1]) and 0 <= x <= 4 * (16 * a[0] * a[2] + 4 + a[0])


def test_empty_problems_do_nothing(bl):
    assert call(bl, "bitlinear_forward_gated", FWD, dict(M=0)) == bl.BL_OK
    assert call(bl, "bitlinear_linear_gated", LIN, dict(M=0)) == bl.BL_OK
    assert call(bl, "bitlinear_gated_backward", BWD, dict(M=0, gb=None)) == bl.BL_OK
    assert call(bl, "bitlinear_gated_backward", BWD, dict(F=0)) == bl.BL_OK
    assert call(bl, "bitlinear_checkpoint", KEEP, dict(M=0)) == bl.BL_OK
    assert call(bl, "bitlinear_checkpoint_restore", BACK, dict(M=0)) == bl.BL_OK
    assert call(bl, "bitlinear_backward_weight_codes", WGT, dict(N=0)) == bl.BL_OK
    assert call(bl, "bitlinear_backward_input_segmented", INP, dict(M=0)) == bl.BL_OK


# ---- the binding: CPU tensors of the right shapes get as far as their device ----------
def product(bl, **kw):
    a = dict(xq=torch.zeros(5, 64, dtype=torch.int8), scale=torch.ones(5), packed=torch.zeros(16, 16, dtype=torch.uint8),
             gammas=torch.ones(2), F=8, K=64)
    return bl.bitlinear_forward_gated(**{**a, **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(xq=torch.zeros(5, 64)), "xq"), (dict(xq=torch.zeros(64, dtype=torch.int8)), "xq"), (dict(K=63), "xq"),
    (dict(scale=torch.ones(4)), "scale"), (dict(packed=torch.zeros(8, 16, dtype=torch.uint8)), "packed"),
    (dict(packed=torch.zeros(16, 32, dtype=torch.uint8)), "packed"), (dict(gammas=torch.ones(1)), "gammas"),
    (dict(gammas=torch.ones(2).double()), "gammas"), (dict(gammas=torch.ones(4)[::2]), "gammas"), (dict(F=9), "packed"),
    (dict(layout="3bit"), "layout"), (dict(bias=torch.ones(8)), "bias"), (dict(bias=torch.ones(16).half()), "bias"),
    (dict(act="swish"), "act"), (dict(out_dtype=torch.float16), "out_dtype"), (dict(y=torch.ones(5, 16)), "y has"),
    (dict(y=torch.ones(5, 8), out_dtype=BF16), "y is"), (dict(z=torch.ones(5, 8)), "z has"),
    (dict(z=torch.ones(5, 16, dtype=BF16)), "z is"), (dict(kept=torch.ones(10, 8)), "kept"),
    (dict(kept=(torch.ones(10, 8), torch.ones(10, 1))), "kept.codes"),
    (dict(kept=(torch.zeros(5, 16, dtype=torch.int8), torch.ones(5, 1))), "kept.codes"),
    (dict(kept=(torch.zeros(10, 8, dtype=torch.int8), torch.ones(10, 2))), "kept.scale"),
    (dict(kept=(torch.zeros(10, 8, dtype=torch.int8),)), "kept"), ({}, "cpu"), (dict(kept=True, z=True), "cpu")])
def test_binding_refuses_product_arguments(bl, kw, word):
    with pytest.raises(bl.BitLinearError, match=word):
        product(bl, **kw)


def test_binding_refuses_fused_arguments(bl):
    w = (torch.zeros(16, 16, dtype=torch.uint8), torch.ones(2), 8)
    for x, word in ((torch.ones(5), "x is"), (torch.ones(2, 64).half(), "x is"), (torch.ones(64, 2).t(), "contiguous"),
                    (torch.ones(2, 64), "cpu")):
        with pytest.raises(bl.BitLinearError, match=word):
            bl.linear_gated(x, *w)
        with pytest.raises(bl.BitLinearError, match=word):
            bl.bitlinear_linear_gated(x, *w)
    with pytest.raises(bl.BitLinearError, match="cpu"):  # a checkpoint takes the two-launch way at any M
        bl.linear_gated(torch.ones(2, 64), *w, kept=True)


@pytest.mark.parametrize("kw,word", [
    (dict(grad_y=torch.ones(5)), "grad_y"), (dict(z=torch.ones(5, 8)), "z has"), (dict(z=torch.ones(5, 16).half()), "z is"),
    (dict(z=(torch.zeros(10, 8, dtype=torch.int8), torch.ones(5, 1))), "kept.scale"),
    (dict(z=(torch.zeros(10, 8), torch.ones(10, 1))), "kept.codes"), (dict(act="swish"), "act"),
    (dict(grad_bias=torch.ones(8)), "grad_bias"), (dict(grad_z=torch.ones(5, 8)), "grad_z"),
    (dict(out_dtype=torch.float16), "out_dtype"), ({}, "cpu")])
def test_binding_refuses_backward_arguments(bl, kw, word):
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_gated_backward(**{**dict(grad_y=torch.ones(5, 8), z=torch.ones(5, 16)), **kw})


def test_binding_refuses_checkpoint_arguments(bl):
    good = bl.Checkpoint(torch.zeros(5, 70, dtype=torch.int8), torch.ones(5, 2))
    for f, word in ((lambda: bl.bitlinear_checkpoint(torch.ones(5)), "x is"),
                    (lambda: bl.bitlinear_checkpoint(torch.ones(5, 70).half()), "x is"),
                    (lambda: bl.bitlinear_checkpoint(torch.ones(70, 5).t()), "contiguous"),
                    (lambda: bl.bitlinear_checkpoint(torch.ones(5, 71), good), "kept.codes"),
                    (lambda: bl.bitlinear_checkpoint(torch.ones(5, 70)), "cpu"),
                    (lambda: bl.bitlinear_checkpoint_restore(torch.ones(5, 70)), "kept"),
                    (lambda: bl.bitlinear_checkpoint_restore((good.codes, torch.ones(5, 1))), "kept.scale"),
                    (lambda: bl.bitlinear_checkpoint_restore((torch.zeros(5, dtype=torch.int8), good.scale)), "kept.codes"),
                    (lambda: bl.bitlinear_checkpoint_restore(good, torch.float16), "out_dtype"),
                    (lambda: bl.bitlinear_checkpoint_restore(good, y=torch.ones(5, 71)), "y has"),
                    (lambda: bl.bitlinear_checkpoint_restore(good), "cpu")):
        with pytest.raises(bl.BitLinearError, match=word):
            f()


@pytest.mark.parametrize("kw,word", [
    (dict(grad_y=torch.ones(5)), "grad_y"), (dict(grad_y=torch.ones(5, 8).half()), "grad_y"),
    (dict(xq=torch.zeros(4, 16, dtype=torch.int8)), "xq"), (dict(xq=torch.zeros(5, 16)), "xq"),
    (dict(xq=torch.zeros(16, dtype=torch.int8)), "xq"), (dict(scale=torch.ones(4)), "scale"),
    (dict(grad_w=torch.ones(16, 8)), "grad_w"), (dict(out_dtype=torch.float16), "out_dtype"),
    (dict(grad_w=torch.ones(8, 16), out_dtype=BF16), "grad_w is"), ({}, "cpu")])
def test_binding_refuses_weight_arguments(bl, kw, word):
    a = dict(grad_y=torch.ones(5, 8), xq=torch.zeros(5, 16, dtype=torch.int8), scale=torch.ones(5))
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_backward_weight_codes(**{**a, **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(grad_y=torch.ones(5, 17)), "17 columns"), (dict(grad_y=torch.ones(5)), "grad_y"), (dict(seg_rows=[8, 9]), "columns"),
    (dict(packed=torch.zeros(15, 16, dtype=torch.uint8)), "packed"), (dict(K=65), "packed"), (dict(gammas=torch.ones(1)), "gammas"),
    (dict(layout="3bit"), "layout"), (dict(out_dtype=torch.float16), "out_dtype"), (dict(grad_x=torch.ones(5, 63)), "grad_x"),
    ({}, "cpu"), (dict(seg_rows=16), "cpu")])
def test_binding_refuses_input_arguments(bl, kw, word):
    a = dict(grad_y=torch.ones(5, 16), packed=torch.zeros(16, 16, dtype=torch.uint8), gammas=torch.ones(2), seg_rows=[8, 8], K=64)
    with pytest.raises(bl.BitLinearError, match=word):
        bl.bitlinear_backward_input_segmented(**{**a, **kw})


def test_binding_refuses_a_stream_of_another_device(bl):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    st, h, q = Stream(), torch.ones(2, 64), torch.zeros(2, 64, dtype=torch.int8)
    w = (torch.zeros(16, 16, dtype=torch.uint8), torch.ones(2), 8)
    kept = bl.Checkpoint(q, torch.ones(2, 1))
    for f in (lambda: bl.bitlinear_forward_gated(q, torch.ones(2), *w, 64, stream=st), lambda: bl.linear_gated(h, *w, stream=st),
              lambda: bl.bitlinear_linear_gated(h, *w, stream=st), lambda: bl.bitlinear_gated_backward(h, h, stream=st),
              lambda: bl.bitlinear_checkpoint(h, stream=st), lambda: bl.bitlinear_checkpoint_restore(kept, stream=st),
              lambda: bl.bitlinear_backward_weight_codes(h, q, torch.ones(2), stream=st),
              lambda: bl.bitlinear_backward_input_segmented(torch.ones(2, 16), w[0], w[1], 16, 64, stream=st)):
        with pytest.raises(bl.BitLinearError, match="stream is of cuda:1"):
            f()


def test_counts_are_read_at_each_call(bl):
    """Rows and widths held in 0-d tensors are the numbers that they are at the call."""
    F, K, rows = torch.tensor(8), torch.tensor(64), [torch.tensor(8), torch.tensor(8)]
    for f, k, word in ((8, 64, "cpu"), (9, 64, "packed"), (8, 64, "cpu")):
        F.fill_(f)
        with pytest.raises(bl.BitLinearError, match=word):
            product(bl, F=F)
    for k, word in ((64, "cpu"), (128, "packed"), (64, "cpu")):
        K.fill_(k)
        with pytest.raises(bl.BitLinearError, match=word):
            product(bl, xq=torch.zeros(5, k, dtype=torch.int8), K=K)
        with pytest.raises(bl.BitLinearError, match=word):
            bl.bitlinear_backward_input_segmented(torch.ones(5, 16), torch.zeros(16, 16, dtype=torch.uint8), torch.ones(2),
                                                  rows, K)
    rows[0] += 1
    with pytest.raises(bl.BitLinearError, match="16 columns for 17"):
        bl.bitlinear_backward_input_segmented(torch.ones(5, 16), torch.zeros(16, 16, dtype=torch.uint8), torch.ones(2), rows, 64)


def test_workspace_of_the_largest_numbers_is_none(bl):
    """2 M may not overflow on its way to the limit."""
    for big in (2 ** 62, 2 ** 62 + 1, 2 ** 63 - 1):
        assert bl.bitlinear_gated_backward_workspace_bytes(big, 8) == 0
        assert bl.bitlinear_gated_backward_workspace_bytes(8, big) == 0
