"""Refusals of the grouped products, the INT8 products and SwiGLU: the C ABI's codes on the host, before
any CUDA call (the pointers are never dereferenced), and the binding's checks on CPU tensors."""
import ctypes
import os

import pytest
import torch

import group_limited_routing_router_b200 as bm
from group_limited_routing_router_b200 import build as bm_build

P, MIS = 4096, 4104
BF, HF, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    bm_build.build()
    return bm.lib()


# each call with its arguments by name, in order; the last is the stream
def mm(**kw):
    a = dict(E=4, R=100, K=128, N=64, dtype=BF, x=P, ldx=128, off=P, w=P, out_dtype=BF, out=P, ldo=64, s=None)
    return a | kw


def dgrad(**kw):
    a = dict(E=4, R=100, K=128, N=64, dtype=BF, dy=P, ldy=64, off=P, w=P, out_dtype=BF, dx=P, ldx=128, s=None)
    return a | kw


def wgrad(**kw):
    a = dict(E=4, R=100, K=128, N=64, dtype=BF, dy=P, ldy=64, x=P, ldx=128, off=P, out_dtype=BF, dw=P, acc=0,
             ws=None, n=0, s=None)
    return a | kw


def i8(**kw):
    a = dict(E=4, R=100, K=128, N=64, q=P, rs=P, off=P, w=P, cs=P, out_dtype=BF, out=P, ldo=64, s=None)
    return a | kw


def quant(**kw):
    return dict(R=10, K=64, dtype=BF, x=P, ldx=64, q=P, scale=P, s=None) | kw


def swiglu(**kw):
    return dict(R=10, I=64, dtype=BF, g=P, ldg=64, u=P, ldu=64, h=P, ldh=64, s=None) | kw


def swiglu_backward(**kw):
    return dict(R=10, I=64, dtype=BF, dh=P, lddh=64, g=P, ldg=64, u=P, ldu=64, dg=P, lddg=64, du=P, lddu=64,
                s=None) | kw


def swiglu_i8(**kw):
    return dict(R=10, I=64, dtype=BF, g=P, ldg=64, u=P, ldu=64, q=P, scale=P, s=None) | kw


NAMES = {mm: "grouped_mm", dgrad: "grouped_mm_dgrad", wgrad: "grouped_mm_wgrad", i8: "grouped_mm_i8",
         quant: "quant_i8_rows", swiglu: "swiglu", swiglu_backward: "swiglu_backward", swiglu_i8: "swiglu_i8"}
PRODUCTS = (mm, dgrad, wgrad, i8)
CFG, NULL, MISAL, SMALL, ARG = (bm.ERR_INVALID_CONFIG, bm.ERR_NULL, bm.ERR_MISALIGNED,
                                bm.ERR_WORKSPACE_TOO_SMALL, bm.ERR_INVALID_ARG)


def call(L, f, **kw):
    return getattr(L, "beam_moe_" + NAMES[f])(*f(**kw).values())


@pytest.mark.parametrize("f", PRODUCTS)
def test_shapes(L, f):
    for bad in (dict(E=0), dict(E=257), dict(K=0), dict(K=100), dict(N=4), dict(N=65544), dict(K=65552)):
        assert call(L, f, **bad) == CFG, bad
    assert call(L, f, R=-1) == ARG and call(L, f, R=(1 << 24) + 1) == ARG
    assert call(L, f, E=2, off=None) == NULL  # only one group can do without offsets
    assert call(L, f, off=4100) == MISAL
    assert call(L, f, out_dtype=7) == ARG
    if f is not wgrad:  # wgrad writes zeros there
        assert call(L, f, R=0) == bm.OK


def test_int8_widths_are_whole_16_byte_pieces(L):
    assert call(L, i8, K=136) == CFG and call(L, i8, N=72) == CFG
    for f in (mm, dgrad, wgrad):
        assert call(L, f, K=132) == CFG and call(L, f, N=68) == CFG


@pytest.mark.parametrize("f", (mm, dgrad, wgrad))
def test_types(L, f):
    assert call(L, f, dtype=F32) == ARG and call(L, f, dtype=-1) == ARG
    assert call(L, f, dtype=BF, out_dtype=HF) == ARG and call(L, f, dtype=HF, out_dtype=BF) == ARG


@pytest.mark.parametrize("f,names", [(mm, "x w out"), (dgrad, "dy w dx"), (wgrad, "dy x dw"), (i8, "q w out"),
                                     (quant, "x q"), (swiglu, "g u h"), (swiglu_backward, "dh g u dg du"),
                                     (swiglu_i8, "g u q")])
def test_pointers(L, f, names):
    for n in names.split():
        assert call(L, f, **{n: None}) == NULL, n
        assert call(L, f, **{n: MIS}) == MISAL, n


@pytest.mark.parametrize("f,names", [(i8, "rs cs"), (quant, "scale"), (swiglu_i8, "scale")])
def test_scale_pointers(L, f, names):
    for n in names.split():
        assert call(L, f, **{n: None}) == NULL and call(L, f, **{n: 4098}) == MISAL, n


@pytest.mark.parametrize("f,ld,width", [(mm, "ldx", 128), (mm, "ldo", 64), (dgrad, "ldy", 64), (dgrad, "ldx", 128),
                                        (wgrad, "ldy", 64), (wgrad, "ldx", 128), (i8, "ldo", 64), (quant, "ldx", 64),
                                        (swiglu, "ldg", 64), (swiglu, "ldu", 64), (swiglu, "ldh", 64),
                                        (swiglu_backward, "lddh", 64), (swiglu_backward, "lddg", 64),
                                        (swiglu_backward, "lddu", 64), (swiglu_i8, "ldg", 64),
                                        (swiglu_i8, "ldu", 64)])
def test_row_strides(L, f, ld, width):
    """Below the width, off the 16-byte boundaries, beyond 2^32."""
    for bad in (width - 8, 0, -width, width + 4, (1 << 32) + 8):
        assert call(L, f, **{ld: bad}) == ARG, bad


@pytest.mark.parametrize("f,width", [(quant, "K"), (swiglu, "I"), (swiglu_backward, "I"), (swiglu_i8, "I")])
def test_row_calls(L, f, width):
    for bad in (0, 4, 60, 65544):
        assert call(L, f, **{width: bad}) == CFG
    assert call(L, f, dtype=3) == ARG and call(L, f, R=-1) == ARG
    assert call(L, f, R=0) == bm.OK


def test_wgrad_workspace(L):
    size = L.beam_moe_grouped_mm_wgrad_workspace_size
    assert size(256, 32768, 5120, 2560) == 0 and size(1, 100, 128, 64) == 0
    assert size(0, 100, 128, 64) == 0 and size(1, -1, 128, 64) == 0 and size(1, 100, 100, 64) == 0
    need = size(1, 20000, 320, 192)
    assert need > 0 and need % (320 * 192 * 4) == 0
    big = dict(E=1, R=20000, K=320, N=192, ldx=320, ldy=192, off=None)
    assert call(L, wgrad, **big) == NULL
    assert call(L, wgrad, **big, ws=P, n=need - 1) == SMALL
    assert call(L, wgrad, **big, ws=MIS, n=need) == MISAL


def test_accumulation_is_fp32_only(L):
    assert call(L, wgrad, acc=1, out_dtype=BF) == ARG
    assert call(L, wgrad, dw=None, R=0) == NULL


def test_binding_refuses_cpu_tensors(L):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    for f in (lambda: bm.grouped_mm(x, w), lambda: bm.grouped_mm_dgrad(x, w), lambda: bm.grouped_mm_wgrad(x, x),
              lambda: bm.quant_i8_rows(x), lambda: bm.swiglu(x, x), lambda: bm.swiglu_backward(x, x, x),
              lambda: bm.swiglu_i8(x, x), lambda: bm.grouped_mm_i8(x.to(torch.int8), x[:, 0], w, w),
              lambda: bm.grouped_mm_i8(None, None, None, None)):
        with pytest.raises(TypeError):
            f()


def test_no_load_is_non_coherent():
    """Kernels that are launched while the stream's last one still runs live while it writes what they read (the
    quantiser's row scales): non-coherent loads are not for such data.  The join kernel is launched after it."""
    csrc = os.path.join(os.path.dirname(bm.__file__), "csrc")
    for name in ("ragged.cuh", "swiglu.cuh"):
        with open(os.path.join(csrc, name)) as f:
            code = f.read()
        assert "launch_after(ragged_join" not in code and "wait_for_stream();" in code
        kernels = code.split("void __launch_bounds__(256) ragged_join_kernel")[0]
        for load in ("__ldg", "ld.global.nc", "__restrict__", "__ldlu", "__ldcv"):
            assert load not in kernels, (name, load)


def test_cleared_rows_are_released_to_the_cluster():
    """The weight gradient's helper writes shared memory that the other CTA's products read: a release at cluster
    scope on its side, an acquire on theirs."""
    with open(os.path.join(os.path.dirname(bm.__file__), "csrc", "ragged.cuh")) as f:
        code = f.read()
    helper = code.split("helper: clears the rows behind the group")[1].split("epilogue: lanes = rows n")[0]
    assert "mbar_release_smem(full_lead" in helper and "mbar_arrive_async" not in helper
    # it lets items pass that have nothing to clear, so what it waits for may be many items away: a call of 640000 rows
    # by 65536 x 65536 runs for some 4 s, the limit of one wait is 2e9 cycles
    passes = "".join(helper.split())
    assert "if(!needs_clearing(v)){limit+=timeout;continue;}" in passes
    assert "mbar_wait(&tail[stage],phase,limit))break;limit=timeout;" in passes
    issuer = code.split("ragged_wgrad_kernel(")[1].split("MMA issuer for the pair")[1].split("helper: clears")[0]
    assert "if (needs_clearing(it.rows - kb * 64)) acquire_smem();" in issuer


def test_partial_sums_are_released_to_the_cluster():
    """The split kernel's CTAs write their partial sums into one another's shared memory: where the last item's were
    read, and where the new ones have arrived, the order holds at cluster scope on both sides."""
    with open(os.path.join(os.path.dirname(bm.__file__), "csrc", "ragged.cuh")) as f:
        code = f.read()
    split = code.split("ragged_split_kernel(const")[1].split("// ---- wgrad on CTA pairs")[0]
    for bar in ("red_empty, (n_item", "red_full, n_item"):
        behind = split.split("mbar_wait(" + bar)[1].split(";")[1:3]
        assert [s.strip() for s in behind] == ["if (!ok) break", "acquire_smem()"], bar
    assert "mbar_release_smem(mapa_shared(smem_u32(red_empty), lane))" in split and "mbar_arrive_async" not in split


def test_docstrings_say_that_autograd_records_nothing():
    for f in (bm.grouped_mm, bm.grouped_mm_i8, bm.swiglu, bm.quant_i8_rows, bm.swiglu_i8):
        assert "not recorded by autograd" in " ".join(f.__doc__.split()).lower(), f.__name__
