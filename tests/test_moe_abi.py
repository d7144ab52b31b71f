"""CPU: argument checks of the norm, the sort by expert and the way back, and
SwiGLU's gradient: every refusal comes before any HIP call, and the binding
refuses tensors that do not fit."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs

A = 1 << 20       # an aligned address that is never followed
NULL = None
INVALID, SHAPE, MISALIGNED = fp8bs.ERR_INVALID_ARG, fp8bs.ERR_UNSUPPORTED_SHAPE, fp8bs.ERR_MISALIGNED


def norm(x=A, ldx=256, r=2 * A, ldr=256, gamma=A, gt=0, eps=1e-6, T=4, C=256, h=3 * A, ldh=256, q=A, ldq=256, s=A,
         lds=2, y=4 * A, ldy=256, rstd=A):
    return fp8bs.load().fp8bs_rmsnorm_quant_1x128(x, ldx, r, ldr, gamma, gt, eps, T, C, h, ldh, q, ldq, s, lds, y, ldy,
                                                  rstd, NULL)


def norm_bwd(dn=A, lddn=256, dres=2 * A, lddr=256, h=3 * A, ldh=256, gamma=A, gt=1, rstd=A, T=4, C=256, dx=4 * A,
             lddx=256, dgamma=A, ws=A, ws_bytes=1 << 20):
    return fp8bs.load().fp8bs_rmsnorm_bwd(dn, lddn, dres, lddr, h, ldh, gamma, gt, rstd, T, C, dx, lddx, dgamma, ws,
                                          ws_bytes, NULL)


def sort(ids=A, it=1, ldi=8, T=4, k=8, first=0, E=16, M=32, offsets=A, slot=A, ws=NULL, ws_bytes=0):
    return fp8bs.load().fp8bs_moe_sort(ids, it, ldi, T, k, first, E, M, offsets, slot, ws, ws_bytes, NULL)


def gather(src=1, x=A, ldx=256, s_in=A, lds_in=2, T=4, C=256, slot=A, k=8, q=A, ldq=256, s=A, lds=2, y=2 * A, ldy=256,
           M=32):
    return fp8bs.load().fp8bs_moe_gather(src, x, ldx, s_in, lds_in, T, C, slot, k, q, ldq, s, lds, y, ldy, M, NULL)


def dispatch(src=1, x=A, ldx=256, s_in=NULL, lds_in=0, T=4, C=256, ids=A, it=0, ldi=8, k=8, first=0, E=16, offsets=A,
             slot=A, q=A, ldq=256, s=A, lds=2, y=NULL, ldy=0, M=32, ws=NULL, ws_bytes=0):
    return fp8bs.load().fp8bs_moe_dispatch(src, x, ldx, s_in, lds_in, T, C, ids, it, ldi, k, first, E, offsets, slot, q,
                                           ldq, s, lds, y, ldy, M, ws, ws_bytes, NULL)


def combine(y=A, yt=0, ldy=256, M=32, slot=A, w=A, ldw=8, T=4, k=8, N=256, add=2 * A, ldadd=256, out=3 * A, ldo=256):
    return fp8bs.load().fp8bs_moe_combine(y, yt, ldy, M, slot, w, ldw, T, k, N, add, ldadd, out, ldo, NULL)


def combine_bwd(dout=A, lddo=256, y=2 * A, yt=0, ldy=256, slot=A, w=A, ldw=8, T=4, k=8, N=256, q=A, ldq=256, s=A, lds=2,
                dy=3 * A, lddy=256, M=32, dw=A, lddw=8):
    return fp8bs.load().fp8bs_moe_combine_bwd(dout, lddo, y, yt, ldy, slot, w, ldw, T, k, N, q, ldq, s, lds, dy, lddy, M,
                                              dw, lddw, NULL)


def swiglu_bwd(dh=A, lddh=256, g=A, ldg=256, u=A, ldu=256, T=4, I=256, q=A, ldq=512, s=A, lds=4, d=A, ldd=512, h=A,
               ldh=256):
    return fp8bs.load().fp8bs_swiglu_bwd_quant_1x128(dh, lddh, g, ldg, u, ldu, T, I, q, ldq, s, lds, d, ldd, h, ldh, NULL)


REFUSALS = [
    (norm, dict(T=-1), INVALID), (norm, dict(C=0), INVALID), (norm, dict(C=200), SHAPE),
    (norm, dict(C=16512, ldx=16512), SHAPE), (norm, dict(T=1 << 31), SHAPE), (norm, dict(gt=2), INVALID),
    (norm, dict(eps=0.0), INVALID), (norm, dict(eps=-1.0), INVALID), (norm, dict(eps=float("inf")), INVALID),
    (norm, dict(eps=float("nan")), INVALID), (norm, dict(r=NULL), INVALID), (norm, dict(h=NULL), INVALID),
    (norm, dict(q=NULL, s=NULL, y=NULL), INVALID), (norm, dict(q=NULL), INVALID), (norm, dict(s=NULL), INVALID),
    (norm, dict(x=NULL), INVALID), (norm, dict(gamma=NULL), INVALID), (norm, dict(ldx=128), INVALID),
    (norm, dict(ldr=128), INVALID), (norm, dict(ldh=248), INVALID), (norm, dict(ldq=240), INVALID),
    (norm, dict(lds=1), INVALID), (norm, dict(ldy=8), INVALID), (norm, dict(x=A + 8), MISALIGNED),
    (norm, dict(gamma=A + 4), MISALIGNED), (norm, dict(rstd=A + 2), MISALIGNED), (norm, dict(ldx=260), MISALIGNED),
    (norm, dict(h=A, ldh=264), INVALID), (norm, dict(h=2 * A, ldh=264), INVALID),
    (norm_bwd, dict(T=-1), INVALID), (norm_bwd, dict(C=100), SHAPE), (norm_bwd, dict(gt=-1), INVALID),
    (norm_bwd, dict(dn=NULL), INVALID), (norm_bwd, dict(h=NULL), INVALID), (norm_bwd, dict(rstd=NULL), INVALID),
    (norm_bwd, dict(dx=NULL), INVALID), (norm_bwd, dict(T=600, ws=NULL), INVALID), (norm_bwd, dict(T=600, ws_bytes=256 * 1024 - 1), INVALID),
    (norm_bwd, dict(ws=A + 8), MISALIGNED), (norm_bwd, dict(dgamma=A + 4), MISALIGNED),
    (norm_bwd, dict(dx=A), INVALID), (norm_bwd, dict(dx=3 * A), INVALID),
    (norm_bwd, dict(dx=2 * A, lddx=264), INVALID), (norm_bwd, dict(lddr=128), INVALID),
    (sort, dict(it=2), INVALID), (sort, dict(T=-1), INVALID), (sort, dict(k=0), INVALID), (sort, dict(k=65, ldi=65), SHAPE),
    (sort, dict(E=0), INVALID), (sort, dict(E=1025), SHAPE), (sort, dict(first=-1), INVALID), (sort, dict(M=-1), INVALID),
    (sort, dict(M=1 << 31), SHAPE), (sort, dict(T=(1 << 30) // 8 + 1), SHAPE), (sort, dict(ldi=7), INVALID),
    (sort, dict(ids=NULL), INVALID), (sort, dict(offsets=NULL), INVALID), (sort, dict(slot=NULL), INVALID),
    (sort, dict(ids=A + 4), MISALIGNED), (sort, dict(it=0, ids=A + 2), MISALIGNED), (sort, dict(slot=A + 1), MISALIGNED),
    (sort, dict(T=5000), INVALID), (sort, dict(T=5000, ws=A, ws_bytes=40 * 16 * 4 - 1), INVALID),
    (gather, dict(src=2), INVALID), (gather, dict(src=0), INVALID), (gather, dict(src=0, y=NULL, s_in=NULL), INVALID),
    (gather, dict(q=NULL, s=NULL, y=NULL), INVALID), (gather, dict(q=NULL), INVALID), (gather, dict(x=NULL), INVALID),
    (gather, dict(slot=NULL), INVALID), (gather, dict(C=100), SHAPE), (gather, dict(C=-128), INVALID),
    (gather, dict(k=65), SHAPE), (gather, dict(T=1 << 31), SHAPE), (gather, dict(M=1 << 31), SHAPE),
    (gather, dict(ldx=128), INVALID), (gather, dict(ldq=264), MISALIGNED), (gather, dict(y=A + 2), MISALIGNED),
    (dispatch, dict(src=2), INVALID), (dispatch, dict(it=5), INVALID), (dispatch, dict(q=NULL, s=NULL), INVALID),
    (dispatch, dict(C=64), SHAPE), (dispatch, dict(E=2000), SHAPE), (dispatch, dict(T=5000), INVALID),
    (dispatch, dict(x=NULL), INVALID), (dispatch, dict(src=0), INVALID), (dispatch, dict(M=-1), INVALID),
    (dispatch, dict(T=0, C=64), SHAPE), (dispatch, dict(M=0, src=2), INVALID),
    (combine, dict(yt=2), INVALID), (combine, dict(y=NULL), INVALID), (combine, dict(slot=NULL), INVALID),
    (combine, dict(out=NULL), INVALID), (combine, dict(k=0), INVALID), (combine, dict(k=65, ldw=65), SHAPE),
    (combine, dict(N=192), SHAPE), (combine, dict(ldw=7), INVALID), (combine, dict(ldy=128), INVALID),
    (combine, dict(out=A), INVALID), (combine, dict(out=2 * A, ldo=264), INVALID), (combine, dict(w=A + 2), MISALIGNED),
    (combine, dict(yt=1, ldy=254), INVALID), (combine, dict(M=-1), INVALID),
    (combine_bwd, dict(w=NULL), INVALID), (combine_bwd, dict(y=NULL), INVALID), (combine_bwd, dict(slot=NULL), INVALID),
    (combine_bwd, dict(q=NULL, s=NULL, dy=NULL, dw=NULL), INVALID), (combine_bwd, dict(s=NULL), INVALID),
    (combine_bwd, dict(dy=A), INVALID), (combine_bwd, dict(dy=2 * A), INVALID), (combine_bwd, dict(N=100), SHAPE),
    (combine_bwd, dict(lddw=7), INVALID), (combine_bwd, dict(dout=A + 8), MISALIGNED), (combine_bwd, dict(yt=9), INVALID),
    (swiglu_bwd, dict(T=-1), INVALID), (swiglu_bwd, dict(I=0), INVALID), (swiglu_bwd, dict(I=100), SHAPE),
    (swiglu_bwd, dict(q=NULL, s=NULL, d=NULL, h=NULL), INVALID), (swiglu_bwd, dict(q=NULL), INVALID),
    (swiglu_bwd, dict(ldq=256), INVALID), (swiglu_bwd, dict(lds=2), INVALID), (swiglu_bwd, dict(ldd=256), INVALID),
    (swiglu_bwd, dict(dh=NULL), INVALID), (swiglu_bwd, dict(u=A + 2), MISALIGNED), (swiglu_bwd, dict(ldg=260), MISALIGNED),
]


@pytest.mark.parametrize("call,args,expect", REFUSALS,
                         ids=[f"{c.__name__}-{'-'.join(f'{k}={v}' for k, v in a.items())}" for c, a, _ in REFUSALS])
def test_refusals(call, args, expect):
    assert call(**args) == expect


@pytest.mark.parametrize("call", [norm, norm_bwd, sort, gather, dispatch, combine, combine_bwd, swiglu_bwd])
def test_valid_arguments_reach_the_device(call):
    if torch.cuda.is_available():
        pytest.skip("addresses here are never followed")
    args = dict(y=NULL) if call is gather else {}
    assert call(**args) == fp8bs.ERR_NO_DEVICE
    if call is gather:
        assert call(src=0, y=NULL) == fp8bs.ERR_NO_DEVICE


@pytest.mark.parametrize("call,args", [(norm, dict(T=0)), (norm_bwd, dict(T=0, dgamma=NULL)), (gather, dict(T=0)),
                                       (gather, dict(M=0, q=NULL, s=NULL, y=NULL)), (combine, dict(T=0)),
                                       (combine_bwd, dict(T=0)), (combine_bwd, dict(M=0, dw=NULL)), (swiglu_bwd, dict(T=0))])
def test_nothing_to_do(call, args):
    nothing = {k: NULL for k in ("x", "r", "dh", "dn", "dout", "h", "slot") if k in call.__code__.co_varnames}
    assert call(**{**nothing, **args}) == fp8bs.OK


def test_working_memory():
    assert fp8bs.fp8bs_moe_sort_ws(1024, 8, 256) == 0
    assert fp8bs.fp8bs_moe_sort_ws(1025, 8, 256) == 9 * 256 * 4
    assert all(0 < fp8bs.fp8bs_moe_sort_ws(t, 8, e) <= 1 << 18 for t in (1 << 13, 1 << 20, 1 << 27)
               for e in (1, 64, 65, 256, 257, 1024))
    assert fp8bs.fp8bs_moe_sort_ws(0, 8, 16) == 0
    for bad in ((-1, 8, 16), (4, 0, 16), (4, 65, 16), (4, 8, 0), (4, 8, 1025), (1 << 28, 8, 16)):
        assert fp8bs.fp8bs_moe_sort_ws(*bad) == -1
    assert fp8bs.fp8bs_rmsnorm_bwd_ws(512, 256) == 0
    assert fp8bs.fp8bs_rmsnorm_bwd_ws(600, 256) == 256 * 256 * 4
    assert all(0 < fp8bs.fp8bs_rmsnorm_bwd_ws(1 << 30, 128 * g) < 1 << 25 for g in range(1, 129))
    assert fp8bs.fp8bs_rmsnorm_bwd_ws(0, 256) == 0
    for bad in ((-1, 256), (4, 0), (4, 100), (4, 16512), (1 << 31, 256)):
        assert fp8bs.fp8bs_rmsnorm_bwd_ws(*bad) == -1


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


B = fp8bs
BINDING = [
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(128), 1e-6, None, u8(4, 256), torch.zeros(4, 2), None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(256).half(), 1e-6, None, u8(4, 256), torch.zeros(4, 2), None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), bf16(4, 256), bf16(256), 1e-6, None, u8(4, 256), torch.zeros(4, 2), None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(256), 1e-6, None, u8(3, 256), torch.zeros(4, 2), None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(256), 1e-6, None, u8(4, 256), None, None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(256), 1e-6, None, None, None, None, None),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256), None, bf16(256), 1e-6, None, None, None, bf16(4, 256), torch.zeros(3)),
    lambda: B.fp8bs_rmsnorm_quant_1x128(bf16(4, 256).float(), None, bf16(256), 1e-6, None, None, None, bf16(4, 256), None),
    lambda: B.fp8bs_rmsnorm_bwd(bf16(4, 256), None, bf16(4, 256), bf16(256), torch.zeros(3), bf16(4, 256), None, None),
    lambda: B.fp8bs_rmsnorm_bwd(bf16(4, 128), None, bf16(4, 256), bf16(256), torch.zeros(4), bf16(4, 256), None, None),
    lambda: B.fp8bs_rmsnorm_bwd(bf16(4, 256), bf16(3, 256), bf16(4, 256), bf16(256), torch.zeros(4), bf16(4, 256), None, None),
    lambda: B.fp8bs_rmsnorm_bwd(bf16(4, 256), None, bf16(4, 256), bf16(256), torch.zeros(4), bf16(4, 256), torch.zeros(255), u8(9999)),
    lambda: B.fp8bs_moe_sort(i32(4, 2).short(), 0, 8, i32(9), i32(4, 2), None),
    lambda: B.fp8bs_moe_sort(i32(4, 2), 0, 8, i32(9), i32(4, 3), None),
    lambda: B.fp8bs_moe_sort(i32(4, 2), 0, 8, i32(1), i32(4, 2), None),
    lambda: B.fp8bs_moe_sort(i32(4, 4)[:, ::2], 0, 8, i32(9), i32(4, 2), None),
    lambda: B.fp8bs_moe_gather(B.SRC_BF16, bf16(4, 256), None, i32(3, 2), u8(8, 256), torch.zeros(8, 2), None),
    lambda: B.fp8bs_moe_gather(B.SRC_BF16, u8(4, 256), None, i32(4, 2), u8(8, 256), torch.zeros(8, 2), None),
    lambda: B.fp8bs_moe_gather(B.SRC_FP8_1x128, u8(4, 256), None, i32(4, 2), u8(8, 256), torch.zeros(8, 2), None),
    lambda: B.fp8bs_moe_gather(B.SRC_BF16, bf16(4, 256), None, i32(4, 2), u8(8, 256), torch.zeros(7, 2), None),
    lambda: B.fp8bs_moe_gather(B.SRC_BF16, bf16(4, 256), None, i32(4, 2), u8(8, 256), torch.zeros(8, 2), bf16(7, 256)),
    lambda: B.fp8bs_moe_dispatch(B.SRC_BF16, bf16(4, 256), None, i32(5, 2), 0, i32(9), i32(5, 2), u8(8, 256), torch.zeros(8, 2), None, None),
    lambda: B.fp8bs_moe_combine(bf16(8, 256), i32(4, 2), torch.zeros(4, 3), None, bf16(4, 256)),
    lambda: B.fp8bs_moe_combine(bf16(8, 256), i32(4, 2), None, bf16(4, 128), bf16(4, 256)),
    lambda: B.fp8bs_moe_combine(bf16(8, 256), i32(4, 2), None, None, bf16(5, 256)),
    lambda: B.fp8bs_moe_combine(bf16(8, 256).half(), i32(4, 2), None, None, bf16(4, 256)),
    lambda: B.fp8bs_moe_combine_bwd(bf16(4, 256), None, i32(4, 2), torch.zeros(4, 2), None, None, None, None),
    lambda: B.fp8bs_moe_combine_bwd(bf16(4, 256), bf16(7, 256), i32(4, 2), torch.zeros(4, 2), u8(8, 256), torch.zeros(8, 2), None, torch.zeros(4, 2)),
    lambda: B.fp8bs_moe_combine_bwd(bf16(4, 256), None, i32(4, 2), None, u8(8, 256), torch.zeros(8, 2), None, None),
    lambda: B.fp8bs_moe_combine_bwd(bf16(4, 256), None, i32(4, 2), torch.zeros(4, 2), u8(8, 256), torch.zeros(8, 2), None, torch.zeros(4, 2)),
    lambda: B.fp8bs_swiglu_bwd_quant_1x128(bf16(4, 256), bf16(4, 256), bf16(4, 256), u8(4, 256), torch.zeros(4, 4), None, None),
    lambda: B.fp8bs_swiglu_bwd_quant_1x128(bf16(4, 256), bf16(4, 256), bf16(4, 128), None, None, bf16(4, 512), None),
    lambda: B.fp8bs_swiglu_bwd_quant_1x128(bf16(4, 256), bf16(4, 256), bf16(4, 256), None, None, None, None),
    # tensors that fit, but lie on the host
    lambda: B.rmsnorm_quant_1x128(bf16(4, 256), bf16(256)),
    lambda: B.rmsnorm_bwd(bf16(4, 256), bf16(4, 256), bf16(256), torch.zeros(4)),
    lambda: B.moe_sort(i32(4, 2), 8),
    lambda: B.moe_gather(bf16(4, 256), i32(4, 2)),
    lambda: B.moe_dispatch(bf16(4, 256), i32(4, 2), 8),
    lambda: B.moe_combine(bf16(8, 256), i32(4, 2)),
    lambda: B.moe_combine_bwd(bf16(4, 256), i32(4, 2), torch.zeros(4, 2)),
    lambda: B.swiglu_bwd_quant_1x128(bf16(4, 256), bf16(4, 256), bf16(4, 256)),
]


@pytest.mark.parametrize("call", BINDING)
def test_binding_refuses(call):
    with pytest.raises(ValueError):
        call()


def test_other_devices_are_refused(monkeypatch):
    """The kernels run on the current device; a tensor of another one is refused."""
    class On:
        is_cuda = True

        def __init__(self, index):
            self.device = self.index = index

        def data_ptr(self):
            return A

        def get_device(self):
            return self.index

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    B._here(On(1), None, On(1))
    B._here(None)
    for tensors in ((On(0),), (On(1), None, On(2))):
        with pytest.raises(ValueError, match="current device"):
            B._here(*tensors)
