"""The grouped products' entry points on the host: what they refuse before any
device call, and the binding's own checks.  CPU only."""
import pytest
import torch

from dense_fp32_gemm_f32_amd import binding

# Pointers that are never dereferenced: these calls fail validation first.
A, B, C, D, E, F, G, H, I = (0x100000000 * (i + 1) for i in range(9))
BIG = 2 ** 31 - 2 ** 16 + 1
INVALID_DIM, INVALID_LD, NULL_PTR, ALIAS, POINTER, INVALID_ARG = 1, 2, 3, 4, 9, 10


def group_rows(**kw):
    a = dict(n=100, groups=8, per_row=1, index=A, offsets=B, order=C, rows=D)
    a.update(kw)
    return binding.gemm_f32_group_rows(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), INVALID_DIM), (dict(n=BIG), INVALID_DIM), (dict(groups=-1), INVALID_DIM),
    (dict(groups=1025), INVALID_DIM), (dict(per_row=0), INVALID_ARG),
    (dict(per_row=-3), INVALID_ARG), (dict(index=0), NULL_PTR), (dict(offsets=0), NULL_PTR),
    (dict(n=0, offsets=0), NULL_PTR), (dict(order=0), NULL_PTR),
    (dict(index=A + 2), POINTER), (dict(rows=D + 1), POINTER), (dict(offsets=B + 3), POINTER),
    (dict(order=A + 396), ALIAS), (dict(rows=C), ALIAS), (dict(offsets=C - 32), ALIAS),
])
def test_group_rows_refusals(change, code):
    assert group_rows(**change) == code


def test_adjacent_arrays_are_not_aliases():
    assert group_rows(order=A + 400) not in (ALIAS, POINTER, NULL_PTR)
    assert group_rows(offsets=C - 36) not in (ALIAS, POINTER, NULL_PTR)
    assert group_rows(rows=0) not in (ALIAS, POINTER, NULL_PTR)


def grouped(**kw):
    a = dict(transB=0, rows=100, N=24, K=40, groups=4, offsets=A, alpha=1.0, A=B, lda=40,
             rowsA=100, indexA=0, B=C, ldb=24, strideB=960, beta=0.0, C=D, ldc=24, rowsC=100,
             indexC=0, bias=0, strideBias=0, act=0)
    a.update(kw)
    return binding.gemm_f32_grouped(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID_DIM), (dict(N=-1), INVALID_DIM), (dict(K=-1), INVALID_DIM),
    (dict(N=BIG, ldb=BIG, ldc=BIG), INVALID_DIM), (dict(groups=1025), INVALID_DIM),
    (dict(rowsA=99), INVALID_DIM), (dict(rowsC=99), INVALID_DIM),
    (dict(rowsA=-1, indexA=E), INVALID_DIM),
    (dict(lda=39), INVALID_LD), (dict(ldb=23), INVALID_LD), (dict(ldc=23), INVALID_LD),
    (dict(transB=1, ldb=39), INVALID_LD), (dict(strideB=-1), INVALID_LD),
    (dict(strideBias=-1), INVALID_LD), (dict(strideB=2 ** 60), INVALID_LD),
    (dict(lda=2 ** 55), INVALID_LD),
    (dict(act=2), INVALID_ARG), (dict(act=-1), INVALID_ARG),
    (dict(offsets=0), NULL_PTR), (dict(A=0), NULL_PTR), (dict(B=0), NULL_PTR),
    (dict(C=0), NULL_PTR),
    (dict(offsets=A + 2), POINTER), (dict(A=B + 1), POINTER), (dict(indexA=E + 2), POINTER),
    (dict(indexC=E + 2), POINTER), (dict(bias=E + 2), POINTER),
    (dict(C=B + 4 * 40 * 100 - 4), ALIAS), (dict(C=C), ALIAS),
    (dict(C=C + 4 * (3 * 960 + 39 * 24 + 23)), ALIAS), (dict(offsets=D + 400), ALIAS),
    (dict(indexA=D + 400), ALIAS), (dict(indexC=D + 4 * 2399), ALIAS),
    (dict(bias=D, strideBias=24), ALIAS),
])
def test_grouped_refusals(change, code):
    assert grouped(**change) == code


def test_grouped_without_work_succeeds_without_a_device():
    assert grouped(rows=0, rowsA=0, rowsC=0, A=0, C=0) == 0
    assert grouped(N=0, ldb=1, ldc=1) == 0
    assert grouped(groups=0) == 0


def wgrad(**kw):
    a = dict(rows=100, M=24, N=40, groups=4, offsets=A, alpha=1.0, A=B, lda=24, rowsA=100,
             indexA=0, B=C, ldb=40, rowsB=100, indexB=0, beta=0.0, C=D, ldc=40, strideC=960)
    a.update(kw)
    return binding.gemm_f32_grouped_wgrad(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID_DIM), (dict(M=-1), INVALID_DIM), (dict(N=BIG), INVALID_DIM),
    (dict(groups=1025), INVALID_DIM), (dict(rowsA=99), INVALID_DIM),
    (dict(rowsB=99), INVALID_DIM), (dict(lda=23), INVALID_LD), (dict(ldb=39), INVALID_LD),
    (dict(ldc=39), INVALID_LD), (dict(strideC=-1), INVALID_LD), (dict(strideC=959), ALIAS),
    (dict(strideC=0), ALIAS), (dict(offsets=0), NULL_PTR), (dict(A=0), NULL_PTR),
    (dict(B=0), NULL_PTR), (dict(C=0), NULL_PTR), (dict(C=D + 2), POINTER),
    (dict(indexB=E + 1), POINTER), (dict(C=B), ALIAS), (dict(C=C + 4), ALIAS),
    (dict(offsets=D + 4 * (4 * 960 - 1)), ALIAS), (dict(indexA=D), ALIAS),
])
def test_wgrad_refusals(change, code):
    assert wgrad(**change) == code


def test_wgrad_without_work_succeeds_without_a_device():
    assert wgrad(groups=0) == 0
    assert wgrad(M=0, lda=1) == 0
    assert wgrad(N=0, ldb=1, ldc=1) == 0


def adapters(**kw):
    a = dict(trans=0, M=100, N=24, K=40, R=8, groups=4, places=90, offsets=A, order=A + 4096,
             scale=A + 8192, X=B, ldx=40, W=C, ldw=24, D=D, ldd=8, strideD=320, U=E, ldu=24,
             strideU=192, bias=F, H=G, ldh=8, Y=H, ldy=24)
    a.update(kw)
    return binding.gemm_f32_adapters(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INVALID_DIM), (dict(R=-1), INVALID_DIM), (dict(places=-1), INVALID_DIM),
    (dict(groups=1025), INVALID_DIM), (dict(ldx=39), INVALID_LD), (dict(ldw=23), INVALID_LD),
    (dict(ldd=7), INVALID_LD), (dict(ldu=23), INVALID_LD), (dict(ldh=7), INVALID_LD),
    (dict(ldy=23), INVALID_LD), (dict(strideD=-1), INVALID_LD), (dict(strideU=-1), INVALID_LD),
    (dict(trans=1, ldw=39), INVALID_LD), (dict(trans=1, ldw=40, ldd=39), INVALID_LD),
    (dict(trans=1, ldw=40, ldd=40, ldu=7), INVALID_LD),
    (dict(X=0), NULL_PTR), (dict(W=0), NULL_PTR), (dict(D=0), NULL_PTR), (dict(U=0), NULL_PTR),
    (dict(H=0), NULL_PTR), (dict(Y=0), NULL_PTR), (dict(offsets=0), NULL_PTR),
    (dict(order=0), NULL_PTR), (dict(order=A + 4098), POINTER), (dict(scale=A + 8193), POINTER),
    (dict(bias=F + 2), POINTER), (dict(H=H), ALIAS), (dict(Y=B), ALIAS), (dict(H=A), ALIAS),
    (dict(Y=E + 4), ALIAS), (dict(H=D), ALIAS), (dict(bias=H + 40), ALIAS),
])
def test_adapters_refusals(change, code):
    assert adapters(**change) == code


def test_adapters_without_rows_succeed_without_a_device():
    assert adapters(M=0, X=0, Y=0) == 0
    assert adapters(N=0, ldw=1, ldu=1, ldy=1, W=0, Y=0) == 0


def test_binding_refuses_tensors_it_cannot_pass():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="GPU"):
        binding.gemm_grouped(x, torch.zeros(2, 8, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="GPU"):
        binding.group_rows(torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(TypeError, match="int32"):
        binding._index(torch.zeros(4, dtype=torch.int64), "index", x.device)
    with pytest.raises(TypeError, match="contiguous"):
        binding._index(torch.zeros(8, dtype=torch.int32)[::2], "index", x.device)
    with pytest.raises(ValueError, match="3 entries"):
        binding._index(torch.zeros(4, dtype=torch.int32), "index", x.device, 3)
    with pytest.raises(ValueError, match="2x8x8"):
        binding._stack(torch.zeros(2, 8, 9), "B", x.device, 2, 8, 8)
    with pytest.raises(TypeError, match="3-D"):
        binding._stack(x, "B", x.device, 2)
    with pytest.raises(TypeError, match="float32"):
        binding._matrix(x.double(), "A", x.device)
    with pytest.raises(ValueError, match="contiguous"):
        binding._matrix(torch.zeros(8, 4).t(), "A", x.device)
    with pytest.raises(ValueError, match="overlap"):
        binding._matrix(torch.zeros(1, 8).expand(4, 8), "A", x.device)
    with pytest.raises(ValueError, match="overlap"):
        binding._matrix(torch.zeros(20).as_strided((4, 8), (3, 1)), "A", x.device)
    with pytest.raises(ValueError, match="must be 4x9"):
        binding._matrix(x, "A", x.device, 4, 9)
    with pytest.raises(ValueError, match="on cuda"):
        binding._matrix(x, "A", torch.device("cuda", 0))
    with pytest.raises(ValueError, match="vector of 4"):
        binding._vector(torch.zeros(5), "scale", x.device, 4)
    with pytest.raises(ValueError, match="bias must be"):
        binding._biases(torch.zeros(3, 4), x.device, 3, 5)
    assert binding._matrix(x[:, 2:5], "A", x.device)[1:] == (8, 4, 3)
    assert binding._matrix(x[:1, :].expand(1, 8), "A", x.device)[1:] == (8, 1, 8)
    assert binding._matrix(torch.zeros(4, 0), "A", x.device)[1:] == (1, 4, 0)
    assert binding._stack(torch.zeros(1, 8, 4).expand(3, 8, 4), "B", x.device, 3)[1:] == \
        (4, 0, 8, 4)


def test_products_refuse_tensors_whose_rows_overlap():
    """An expanded matrix has no pitch: it would be read past its end."""
    class Gpu:   # what _pitch looks at, with the device a GPU tensor reports
        dtype, shape = torch.float32, (4, 8)
        device = torch.device("cuda", 0)
        def __init__(self, *strides):
            self.strides = strides
        def dim(self):
            return 2
        def stride(self, d):
            return self.strides[d]
    assert binding._pitch(Gpu(8, 1), "A") == 8 and binding._pitch(Gpu(11, 1), "A") == 11
    for s0 in (0, 1, 7):
        with pytest.raises(ValueError, match="overlap"):
            binding._pitch(Gpu(s0, 1), "A")
    with pytest.raises(ValueError, match="offsets"):
        binding._groups_of(torch.zeros(0, dtype=torch.int32))


def test_recorded_traffic_still_belongs_to_its_kernels():
    """The grouped products' declarations stay out of the sources that the other
    kernels' counter records are hashed over: a changed hash drops the record."""
    import json
    from pathlib import Path

    from dense_fp32_gemm_f32_amd.prof_summary import source_hash
    records = json.loads((Path(__file__).parent.parent / "profiles" / "traffic.json").read_text())
    assert records
    for kernel, record in records.items():
        assert record["source_sha256"] == source_hash(kernel), kernel
