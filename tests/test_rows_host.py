"""The row operators without a GPU: refusals before any launch, through the C ABI and through the
binding, and the oracle's e4m3 against torch's own conversion."""
import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
apq = pytest.importorskip("any_precision_expert_router_amd",
                          reason="libmoe_apq.so not built (run __graft_entry__.build())")

FAKE = 0x1000   # never dereferenced: every call below must fail validation first, or do nothing
F16, BF16, F32 = 0, 1, 2
BAD, UNSUP, OK = apq.MOE_EINVAL, apq.MOE_EUNSUPPORTED, apq.MOE_OK


def _with(defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return list(args.values())


PERMUTE = dict(x=FAKE, dtype=F16, x_stride=64, T=4, k=2, E=8, H=64, ids=FAKE, offsets=FAKE, pairs=FAKE,
               xs=FAKE, xs_stride=64, rows=FAKE, stream=None)
PERMUTE_BWD = dict(dxs=FAKE, dtype=F16, dxs_stride=64, T=4, k=2, H=64, rows=FAKE, dx=FAKE, dx_stride=64, stream=None)
UNPERMUTE = dict(ys=FAKE, dtype=BF16, ys_stride=64, T=4, k=2, H=64, rows=FAKE, gates=FAKE, add=FAKE, add_stride=64,
                 y=FAKE, y_stride=64, stream=None)
UNPERMUTE_BWD = dict(dy=FAKE, dtype=F32, dy_stride=64, ys=FAKE, ys_stride=64, T=4, k=2, H=64, rows=FAKE, gates=FAKE,
                     dys=FAKE, dys_stride=64, dgates=FAKE, stream=None)
QUANT = dict(x=FAKE, dtype=F16, x_stride=512, M=4, K=256, n_rows=None, q=FAKE, q_stride=256, scales=FAKE, stream=None)
GEMM = dict(a=FAKE, lda=256, a_scales=FAKE, a_rows=8, w=FAKE, w_scales=FAKE, E=4, M=8, N=64, K=256, offsets=FAKE,
            pairs=None, k=1, c=FAKE, dtype=F16, ldc=64, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=9), BAD), (dict(k=0), BAD), (dict(T=-1), BAD), (dict(E=0), BAD), (dict(H=0), BAD), (dict(dtype=3), BAD),
    (dict(dtype=-1), BAD), (dict(x_stride=63), BAD), (dict(xs_stride=63), BAD), (dict(x=None), BAD), (dict(ids=None), BAD),
    (dict(offsets=None), BAD), (dict(pairs=None), BAD), (dict(xs=None), BAD), (dict(rows=None), BAD),
    (dict(x=FAKE + 1), BAD), (dict(xs=FAKE + 2, dtype=F32), BAD), (dict(T=65537), UNSUP), (dict(E=1025), UNSUP),
    (dict(E=64, k=33), UNSUP), (dict(H=(1 << 20) + 1), UNSUP), (dict(x_stride=1 << 41), UNSUP), (dict(T=0), OK),
], ids=str)
def test_permute_refusals(change, code):
    assert apq.lib().moe_permute_tokens(*_with(PERMUTE, **change)) == code
    assert (apq.lib().moe_last_error() == b"") == (code == OK)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), BAD), (dict(k=0), BAD), (dict(k=33), UNSUP), (dict(H=0), BAD), (dict(dtype=7), BAD),
    (dict(dxs_stride=1), BAD), (dict(dx_stride=1), BAD), (dict(dxs=None), BAD), (dict(rows=None), BAD),
    (dict(dx=None), BAD), (dict(dx=FAKE + 1), BAD), (dict(T=0), OK),
], ids=str)
def test_permute_backward_refusals(change, code):
    assert apq.lib().moe_permute_tokens_backward(*_with(PERMUTE_BWD, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), BAD), (dict(k=0), BAD), (dict(k=33), UNSUP), (dict(H=0), BAD), (dict(dtype=7), BAD),
    (dict(ys_stride=1), BAD), (dict(y_stride=1), BAD), (dict(add_stride=1), BAD), (dict(ys=None), BAD),
    (dict(rows=None), BAD), (dict(y=None), BAD), (dict(add=FAKE + 1), BAD), (dict(T=0, add=None, add_stride=0), OK),
], ids=str)
def test_unpermute_refusals(change, code):
    assert apq.lib().moe_unpermute_tokens(*_with(UNPERMUTE, **change)) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), BAD), (dict(k=33), UNSUP), (dict(H=0), BAD), (dict(dtype=7), BAD), (dict(dy_stride=1), BAD),
    (dict(ys_stride=1), BAD), (dict(dys_stride=1), BAD), (dict(dy=None), BAD), (dict(rows=None), BAD),
    (dict(ys=None), BAD), (dict(dys=None, dgates=None), BAD), (dict(dy=FAKE + 2), BAD), (dict(T=0), OK),
], ids=str)
def test_unpermute_backward_refusals(change, code):
    assert apq.lib().moe_unpermute_tokens_backward(*_with(UNPERMUTE_BWD, **change)) == code


@pytest.mark.parametrize("name", ["moe_fp8_quantize", "moe_fp8_quantize_silu"])
@pytest.mark.parametrize("change,code", [
    (dict(M=-1), BAD), (dict(M=(1 << 21) + 1), UNSUP), (dict(K=0), BAD), (dict(K=(1 << 20) + 1), UNSUP),
    (dict(M=1 << 21, K=1 << 19, x_stride=1 << 20, q_stride=1 << 19), UNSUP), (dict(dtype=3), BAD),
    (dict(x_stride=255), BAD), (dict(q_stride=255), BAD), (dict(x=None), BAD), (dict(q=None), BAD),
    (dict(scales=None), BAD), (dict(x=FAKE + 1), BAD), (dict(M=0), OK),
], ids=str)
def test_quantize_refusals(name, change, code):
    assert getattr(apq.lib(), name)(*_with(QUANT, **change)) == code


def test_quantize_silu_needs_both_halves_in_the_row():
    assert apq.lib().moe_fp8_quantize_silu(*_with(QUANT, x_stride=511)) == BAD


@pytest.mark.parametrize("change,code", [
    (dict(E=0), BAD), (dict(E=1025), UNSUP), (dict(M=-1), BAD), (dict(M=(1 << 21) + 1), UNSUP), (dict(N=0), BAD),
    (dict(K=0), BAD), (dict(K=24), UNSUP), (dict(K=(1 << 20) + 16, lda=1 << 21), UNSUP), (dict(lda=240), BAD),
    (dict(lda=264), UNSUP), (dict(lda=(1 << 24) + 16), UNSUP), (dict(pairs=FAKE, a_rows=1 << 16, lda=1 << 16), UNSUP), (dict(ldc=63), BAD), (dict(dtype=3), BAD), (dict(offsets=None), BAD), (dict(a=None), BAD),
    (dict(a_scales=None), BAD), (dict(w=None), BAD), (dict(w_scales=None), BAD), (dict(c=None), BAD),
    (dict(a_rows=7), BAD), (dict(a_rows=0, pairs=FAKE), BAD), (dict(pairs=FAKE, k=0), BAD), (dict(pairs=FAKE, k=33), BAD),
    (dict(a=FAKE + 8), BAD), (dict(w=FAKE + 4), BAD), (dict(c=FAKE + 1), BAD), (dict(M=0), OK),
], ids=str)
def test_gemm_refusals(change, code):
    assert apq.lib().moe_fp8_gemm(*_with(GEMM, **change)) == code


def _refused(word, fn, *args, **kw):
    with pytest.raises(apq.MoeError, match=word) as err:
        fn(*args, **kw)
    assert err.value.code == BAD


def test_binding_refuses_tensors_that_are_not_on_a_gpu_or_of_another_type():
    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    _refused("not on a GPU", apq.moe_permute_tokens, x, i, i, i, x, i)
    _refused("rows are float16", apq.moe_permute_tokens, x.double(), i, i, i, x, i)
    _refused("not on a GPU", apq.moe_permute_tokens_backward, x, i, x)
    _refused("not on a GPU", apq.moe_unpermute_tokens, x, i, None, x)
    _refused("not on a GPU", apq.moe_unpermute_tokens_backward, x, x, i, None, x, None)
    _refused("not on a GPU", apq.moe_fp8_quantize, x, x, x)
    _refused("equally wide", apq.moe_fp8_quantize_silu, torch.zeros(4, 63), x, x)
    _refused("not on a GPU", apq.moe_fp8_gemm, x, x, x, x, x)


def test_oracle_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(oracle.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())
    r = np.random.default_rng(5)
    values = oracle.e4m3_values()[:127]
    v = np.concatenate([values, (values[1:] + values[:-1]) / 2,                     # every value, every tie
                        r.uniform(-448, 448, 4000), r.uniform(-0.02, 0.02, 4000)]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(oracle.e4m3_encode(v.astype(np.float64)), want)
