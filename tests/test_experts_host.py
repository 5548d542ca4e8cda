"""The operators around an expert layer on the host: what their entry points refuse
before any device call, the binding's own checks, and the packing of 4-bit weights.
CPU only."""
import ctypes

import pytest
import torch

from dense_fp32_gemm_f32_amd import binding, q4

# Pointers that are never dereferenced: these calls fail validation first.
A, B, C, D, E, F, G = (0x100000000 * (i + 1) for i in range(7))
BIG = 2 ** 31 - 2 ** 16 + 1
INVALID_DIM, INVALID_LD, NULL_PTR, ALIAS, POINTER, INVALID_ARG = 1, 2, 3, 4, 9, 10


def route(**kw):
    a = dict(tokens=100, experts=32, top=4, logits=A, ldl=32, bias=B, score=0, groups=4,
             group_top=2, group_best=2, renorm=1, scale=1.0, choice=C, weight=D)
    a.update(kw)
    return binding.gemm_f32_route(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID_DIM), (dict(tokens=BIG), INVALID_DIM),
    (dict(experts=-1), INVALID_DIM), (dict(experts=1025, ldl=1025, groups=1), INVALID_DIM),
    (dict(top=-1), INVALID_DIM), (dict(top=65), INVALID_DIM), (dict(groups=0), INVALID_DIM),
    (dict(groups=5), INVALID_DIM), (dict(groups=-4), INVALID_DIM), (dict(groups=64), INVALID_DIM),
    (dict(ldl=31), INVALID_LD), (dict(ldl=2 ** 55), INVALID_LD),
    (dict(score=2), INVALID_ARG), (dict(score=-1), INVALID_ARG),
    (dict(group_top=0), INVALID_ARG), (dict(group_top=5), INVALID_ARG),
    (dict(group_best=0), INVALID_ARG), (dict(group_best=3), INVALID_ARG),
    (dict(logits=0), NULL_PTR), (dict(choice=0), NULL_PTR), (dict(weight=0), NULL_PTR),
    (dict(logits=A + 2), POINTER), (dict(bias=B + 1), POINTER), (dict(choice=C + 2), POINTER),
    (dict(weight=D + 3), POINTER),
    (dict(weight=C + 4 * 399), ALIAS), (dict(choice=A + 4 * 3199), ALIAS),
    (dict(weight=B + 4 * 31), ALIAS), (dict(choice=A - 4 * 399), ALIAS),
])
def test_route_refusals(change, code):
    assert route(**change) == code


def test_route_without_work_succeeds_without_a_device():
    assert route(tokens=0, logits=0, choice=0, weight=0) == 0
    assert route(top=0, choice=0, weight=0) == 0


def test_adjacent_arrays_are_not_aliases():
    assert route(weight=C + 1600) not in (ALIAS, POINTER, NULL_PTR)
    assert route(bias=0, choice=A - 1600) not in (ALIAS, POINTER, NULL_PTR)


def route_grad(**kw):
    a = dict(tokens=100, experts=32, top=4, logits=A, ldl=32, score=1, renorm=0, scale=1.0,
             choice=B, dweight=C, dlogits=D, lddl=32)
    a.update(kw)
    return binding.gemm_f32_route_grad(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID_DIM), (dict(experts=1025, ldl=1025, lddl=1025), INVALID_DIM),
    (dict(top=65), INVALID_DIM), (dict(ldl=31), INVALID_LD), (dict(lddl=31), INVALID_LD),
    (dict(score=7), INVALID_ARG), (dict(logits=0), NULL_PTR), (dict(choice=0), NULL_PTR),
    (dict(dweight=0), NULL_PTR), (dict(dlogits=0), NULL_PTR), (dict(dlogits=D + 2), POINTER),
    (dict(dlogits=A), ALIAS), (dict(dlogits=B + 4 * 399), ALIAS), (dict(dlogits=C), ALIAS),
])
def test_route_grad_refusals(change, code):
    assert route_grad(**change) == code


def test_route_grad_without_work_succeeds_without_a_device():
    assert route_grad(tokens=0) == 0
    assert route_grad(experts=0, ldl=1, lddl=1) == 0


def join(**kw):
    a = dict(tokens=50, top=3, N=24, H=A, ldh=24, weight=B, choice=C, groups=8, beta=0.0, Y=D,
             ldy=24)
    a.update(kw)
    return binding.gemm_f32_join_rows(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID_DIM), (dict(top=-1), INVALID_DIM), (dict(N=-1), INVALID_DIM),
    (dict(groups=1025), INVALID_DIM), (dict(tokens=2 ** 30, top=3), INVALID_DIM),
    (dict(ldh=23), INVALID_LD), (dict(ldy=23), INVALID_LD), (dict(ldy=2 ** 57), INVALID_LD),
    (dict(H=0), NULL_PTR), (dict(weight=0), NULL_PTR), (dict(Y=0), NULL_PTR),
    (dict(H=A + 2), POINTER), (dict(choice=C + 2), POINTER), (dict(Y=D + 1), POINTER),
    (dict(Y=A + 4 * (150 * 24 - 1)), ALIAS), (dict(Y=B), ALIAS), (dict(Y=C + 596), ALIAS),
])
def test_join_refusals(change, code):
    assert join(**change) == code


def test_join_without_work_succeeds_without_a_device():
    assert join(tokens=0) == 0
    assert join(N=0, ldh=1, ldy=1) == 0


def join_grad(**kw):
    a = dict(tokens=50, top=3, N=24, dY=A, lddy=24, H=B, ldh=24, weight=C, choice=D, groups=8,
             dH=E, lddh=24, dweight=F)
    a.update(kw)
    return binding.gemm_f32_join_rows_grad(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), INVALID_DIM), (dict(groups=-1), INVALID_DIM), (dict(lddy=23), INVALID_LD),
    (dict(ldh=23), INVALID_LD), (dict(lddh=23), INVALID_LD), (dict(dY=0), NULL_PTR),
    (dict(H=0), NULL_PTR), (dict(weight=0), NULL_PTR), (dict(dH=0), NULL_PTR),
    (dict(dweight=0), NULL_PTR), (dict(dweight=F + 2), POINTER), (dict(dH=A), ALIAS),
    (dict(dH=B + 4 * 3599), ALIAS), (dict(dweight=E), ALIAS), (dict(dweight=C), ALIAS),
    (dict(dweight=D), ALIAS),
])
def test_join_grad_refusals(change, code):
    assert join_grad(**change) == code


def test_join_grad_without_work_succeeds_without_a_device():
    assert join_grad(tokens=0) == 0
    assert join_grad(top=0) == 0


def q4_dense(**kw):
    a = dict(M=10, N=24, K=100, alpha=1.0, A=A, lda=100, format=0, group=32, codes=B, ldq=50,
             scale_type=0, scale=C, lds=4, zero=D, ldz=4, beta=0.0, C=E, ldc=24, bias=F, act=0)
    a.update(kw)
    return binding.gemm_f32_q4(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INVALID_DIM), (dict(N=-1), INVALID_DIM), (dict(K=BIG), INVALID_DIM),
    (dict(lda=99), INVALID_LD), (dict(ldq=49), INVALID_LD), (dict(lds=3), INVALID_LD),
    (dict(ldz=3), INVALID_LD), (dict(ldc=23), INVALID_LD), (dict(ldq=2 ** 58), INVALID_LD),
    (dict(K=101, lda=101), INVALID_LD),
    (dict(group=0), INVALID_ARG), (dict(group=16), INVALID_ARG), (dict(group=48), INVALID_ARG),
    (dict(group=-32), INVALID_ARG), (dict(group=-2 ** 63), INVALID_ARG),
    (dict(format=2), INVALID_ARG), (dict(format=-1), INVALID_ARG),
    (dict(scale_type=4), INVALID_ARG), (dict(scale_type=-1), INVALID_ARG),
    (dict(format=1), INVALID_ARG), (dict(act=2), INVALID_ARG),
    (dict(A=0), NULL_PTR), (dict(codes=0), NULL_PTR), (dict(scale=0), NULL_PTR),
    (dict(C=0), NULL_PTR),
    (dict(A=A + 2), POINTER), (dict(scale=C + 2), POINTER), (dict(scale=C + 1, scale_type=1),
                                                           POINTER),
    (dict(C=E + 1), POINTER), (dict(bias=F + 2), POINTER),
    (dict(C=A + 4 * 999), ALIAS), (dict(codes=E + 4 * 239 + 3), ALIAS),
    (dict(C=C + 4 * 92), ALIAS), (dict(C=D + 92), ALIAS), (dict(C=F), ALIAS),
])
def test_q4_refusals(change, code):
    assert q4_dense(**change) == code


def test_q4_of_byte_arrays_need_no_alignment():
    for change in (dict(codes=B + 1), dict(zero=D + 3), dict(scale=C + 1, scale_type=3),
                   dict(scale=C + 2, scale_type=2), dict(group=2 ** 62, lds=1, ldz=1),
                   dict(codes=E + 960), dict(zero=0, ldz=0)):
        assert q4_dense(**change) not in (INVALID_DIM, INVALID_LD, NULL_PTR, ALIAS, POINTER,
                                          INVALID_ARG)


def test_q4_without_work_succeeds_without_a_device():
    assert q4_dense(M=0) == 0
    assert q4_dense(N=0, ldc=1) == 0


def q4_grouped(**kw):
    a = dict(rows=100, N=24, K=100, groups=4, offsets=G, alpha=1.0, A=A, lda=100, rowsA=100,
             indexA=0, format=1, group=64, codes=B, ldq=50, strideQ=1200, scale_type=3, scale=C,
             lds=2, strideS=48, zero=0, ldz=0, strideZ=0, beta=0.0, C=E, ldc=24, rowsC=100,
             indexC=0, bias=F, strideBias=24, act=1)
    a.update(kw)
    return binding.gemm_f32_q4_grouped(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID_DIM), (dict(groups=1025), INVALID_DIM), (dict(rowsA=99), INVALID_DIM),
    (dict(rowsC=99), INVALID_DIM), (dict(strideQ=-1), INVALID_LD), (dict(strideS=-1), INVALID_LD),
    (dict(strideBias=-1), INVALID_LD), (dict(strideQ=2 ** 60), INVALID_LD),
    (dict(format=0, zero=D, ldz=2, strideZ=-1), INVALID_LD), (dict(zero=D, ldz=2), INVALID_ARG),
    (dict(offsets=0), NULL_PTR), (dict(offsets=G + 2), POINTER), (dict(indexA=G + 401), POINTER),
    (dict(offsets=E + 400), ALIAS), (dict(indexC=E), ALIAS),
    (dict(C=B + 3 * 1200 + 23 * 50 + 46), ALIAS), (dict(C=C + 3 * 48 + 44), ALIAS),
    (dict(C=F + 4 * 92), ALIAS),
])
def test_q4_grouped_refusals(change, code):
    assert q4_grouped(**change) == code


def test_q4_grouped_without_work_succeeds_without_a_device():
    assert q4_grouped(rows=0, rowsA=0, rowsC=0) == 0
    assert q4_grouped(groups=0) == 0


def table(kind, *values):
    return (kind * len(values))(*values)


def norm(x=(A, B, 0), n=(100, 7, 0), count=3, out=C, clip=None, max_norm=1.0, **kw):
    xs = None if x is None else table(ctypes.c_void_p, *x)
    ns = None if n is None else table(ctypes.c_int64, *n)
    if clip is None:
        return binding.gemm_f32_norm(count, xs, ns, out)
    ys = None if clip == "in place" else table(ctypes.c_void_p, *clip)
    return binding.gemm_f32_clip(count, xs, ns, ys, max_norm, out)


@pytest.mark.parametrize("change,code", [
    (dict(count=-1), INVALID_DIM), (dict(count=2 ** 20 + 1), INVALID_DIM),
    (dict(n=(100, -1, 0)), INVALID_DIM), (dict(n=(2 ** 40 + 1, 7, 0)), INVALID_DIM),
    (dict(x=None), NULL_PTR), (dict(n=None), NULL_PTR), (dict(out=0), NULL_PTR),
    (dict(x=(A, 0, 0)), NULL_PTR), (dict(x=(A, B + 2, 0)), POINTER), (dict(out=C + 2), POINTER),
    (dict(out=A + 396), ALIAS), (dict(out=B), ALIAS),
])
def test_norm_refusals(change, code):
    assert norm(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(count=-1), INVALID_DIM), (dict(max_norm=-1.0), INVALID_ARG),
    (dict(max_norm=float("nan")), INVALID_ARG), (dict(out=0), NULL_PTR),
    (dict(x=(A, A + 396, 0)), ALIAS), (dict(x=(A, A, 0)), ALIAS), (dict(x=(A + 24, A, 0)), ALIAS),
    (dict(clip=(D, 0, 0)), NULL_PTR), (dict(clip=(D, E + 1, 0)), POINTER),
    (dict(clip=(D, D + 396, 0)), ALIAS), (dict(clip=(A + 4, E, 0)), ALIAS),
    (dict(clip=(B, E, 0)), ALIAS), (dict(clip=(D, C, 0)), ALIAS), (dict(out=A + 4), ALIAS),
    (dict(clip=(A, A + 396, 0)), ALIAS),
])
def test_clip_refusals(change, code):
    assert norm(**{"clip": "in place", **change}) == code


def test_arrays_that_may_touch():
    refused = (INVALID_DIM, NULL_PTR, ALIAS, POINTER, INVALID_ARG)
    assert norm(x=(A, A, 0)) not in refused                       # the norm alone only reads
    assert norm(clip="in place", x=(A, A + 400, 0)) not in refused
    assert norm(clip=(A, B, 0)) not in refused                    # each its own, in place
    assert norm(clip=(A + 400, B, 0)) not in refused
    assert norm(clip=(D, E, 0), x=(A, A, 0)) not in refused       # read twice, written apart


# ---- the binding's checks ---------------------------------------------------------

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 8)
    codes, scale = torch.zeros(3, 4, dtype=torch.uint8), torch.ones(3, 1)
    c = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: binding.route(x, 2), lambda: binding.route_grad(c.float(), x, c),
                 lambda: binding.join_rows(x, torch.ones(2, 2)),
                 lambda: binding.join_rows_grad(x[:2], x, torch.ones(2, 2)),
                 lambda: binding.gemm_q4(x, codes, scale),
                 lambda: binding.gemm_q4_grouped(x, codes[None], scale[None], torch.zeros(2).int()),
                 lambda: binding.norm([x]), lambda: binding.clip_norm([x], 1.0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        binding.norm([])


# ---- packing -------------------------------------------------------------------------

@pytest.mark.parametrize("K", [1, 2, 7, 64, 101])
def test_pack_and_unpack(K):
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 16, (3, 5, K), generator=g)
    packed = q4.pack(codes)
    assert packed.shape == (3, 5, (K + 1) // 2) and packed.dtype == torch.uint8
    assert torch.equal(q4.unpack(packed, K).long(), codes)
    assert int(packed[0, 0, 0]) & 15 == int(codes[0, 0, 0])


@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("form", ["symmetric", "zeros", "e2m1"])
@pytest.mark.parametrize("group,K", [(32, 96), (32, 70), (64, 33), (4096, 50)])
def test_quantize_stays_within_half_a_step(kind, form, group, K):
    """Every weight comes back within half the distance of the values beside it (a
    whole step at the ends, where a rounded scale may not reach), and the largest
    weight of a group sets its scale."""
    g = torch.Generator().manual_seed(group + K)
    W = torch.randn(2, 6, K, generator=g)
    W[0, 0] = 0
    fmt = binding.Q4_E2M1 if form == "e2m1" else binding.Q4_INT
    codes, scale, zero = q4.quantize(W, group=group, format=fmt, symmetric=form == "symmetric",
                                     scale_dtype=kind)
    along = (K + group - 1) // group
    assert codes.shape == (2, 6, (K + 1) // 2) and scale.shape == (2, 6, along)
    assert scale.dtype == kind and (zero is None) == (form != "zeros")
    back = q4.dequantize(codes, scale, K, zero=zero, group=group, format=fmt, dtype=torch.float64)
    by = q4.scale_values(scale).double()[..., torch.arange(K) // group]
    # the widest step is 1 scale for whole numbers, 2 for e2m1 (from 4 to 6)
    assert bool(((back - W.double()).abs() <= by * (1.01 if form != "e2m1" else 1.05)).all())
    assert torch.equal(back[0, 0], torch.zeros(K, dtype=torch.float64))


@pytest.mark.parametrize("size", [1e-9, 1e30])
@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_past_the_scale_type(size, symmetric):
    """Groups whose scale fp16 cannot hold: zeros below, the largest scale above."""
    W = torch.linspace(-1, 1, 64).view(2, 32) * size
    codes, scale, zero = q4.quantize(W, group=32, symmetric=symmetric, scale_dtype=torch.float16)
    back = q4.dequantize(codes, scale, 32, zero=zero, group=32)
    assert bool(scale.isfinite().all()) and bool(back.isfinite().all())
    assert bool((back.abs() <= W.abs().max()).all())


def test_dequantize_by_hand():
    codes = q4.pack(torch.tensor([[0, 15, 8, 3]]))
    scale = torch.tensor([[0.5]])
    assert q4.dequantize(codes, scale, 4, group=32).tolist() == [[-4.0, 3.5, 0.0, -2.5]]
    zero = torch.tensor([[3]], dtype=torch.uint8)
    assert q4.dequantize(codes, scale, 4, zero=zero, group=32).tolist() == [[-1.5, 6.0, 2.5, 0.0]]
    e8m0 = torch.tensor([[128]], dtype=torch.uint8)
    assert q4.dequantize(codes, e8m0, 4, group=32, format=binding.Q4_E2M1).tolist() == [
        [0.0, -12.0, 0.0, 3.0]]
    e = q4.scale_values(torch.tensor([0, 1, 127, 254, 255], dtype=torch.uint8))
    assert e[:4].tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 2.0 ** 127] and e[4].isnan()
