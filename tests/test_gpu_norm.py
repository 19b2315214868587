"""RMS norm and SwiGLU with quantised outputs against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from layer_util import DT, FORMS, NORM_DELTA, SILU_DELTA, check_rows, f64, outputs, run_norm
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def made(seed, M, K, dtype, stride=None, std=1.0):
    """Values of a few sizes, as a slice of wider rows that hold NaN elsewhere."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * std * torch.exp(torch.randn(K, generator=g))
    buf = torch.full((M, stride or K), float("nan"), dtype=DT[dtype][1])
    buf[:, :K] = x.to(DT[dtype][1])
    return buf.cuda()


def weight(seed, K, dtype):
    return (1.0 + 0.2 * torch.randn(K, generator=torch.Generator().manual_seed(seed))).to(DT[dtype][1]).cuda()


# every form at the widths where the row's threads change (512, 2048, 4096, 8192, 16384), around them and at the ends
WIDTHS = [128, 384, 512, 640, 2048, 2176, 4096, 4224, 7168, 8192, 8320, 16384, 16512, 65536]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("form", list(FORMS))
def test_norm_forms_and_widths(form, K):
    dtype = "bf16" if K % 256 else "fp16"
    M = 1 if K > 16384 else 5
    note(f"norm {form} {dtype} M={M} K={K}")
    x, r, w = made(1, M, K, dtype), made(2, M, K, dtype, std=2.0), weight(3, K, "fp32" if K % 384 == 0 else dtype)
    total = torch.empty_like(x)
    got = run_norm(form, dtype, x, r, w, M, K, sum_out=total)
    h, y = ol.rms_norm(f64(x), f64(r), f64(w), float(np.float32(1e-6)))
    check_rows(form, dtype, y, NORM_DELTA, *got)
    assert (np.abs(f64(total) - h) <= np.abs(h) * (DT[dtype][2] + 2.0 ** -23) + 2.0 ** -25).all()


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 63, 100, 511, 777, 1999, 4095, 4097, 5001, 16383, 16385, 65535])
@pytest.mark.parametrize("form", ["same", "f8_token", "i8_token"])
def test_norm_odd_widths(form, K):
    dtype = "fp16" if K % 4 == 1 else "bf16"
    M = 1 if K > 16384 else 3
    note(f"norm {form} {dtype} M={M} K={K}")
    x, r, w = made(4, M, K, dtype), made(5, M, K, dtype), weight(6, K, dtype)
    total = torch.empty_like(x)
    got = run_norm(form, dtype, x, r, w, M, K, sum_out=total)
    h, y = ol.rms_norm(f64(x), f64(r), f64(w), float(np.float32(1e-6)))
    check_rows(form, dtype, y, NORM_DELTA, *got)
    assert (np.abs(f64(total) - h) <= np.abs(h) * (DT[dtype][2] + 2.0 ** -23) + 2.0 ** -25).all()


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("M", [1, 3, 4, 5, 130])
def test_norm_rows_and_strides(form, M):
    """Rows inside wider ones (whole and odd strides), no residual, an offset, a larger eps."""
    K = 384
    for stride in (K + 64, K + 5) if form in ("same", "f8_token", "i8_token") else (K + 64, K + 8):
        note(f"norm {form} M={M} K={K} stride={stride}")
        x, w = made(7, M, K, "bf16", stride), weight(8, K, "bf16")
        got = run_norm(form, "bf16", x, None, w, M, K, eps=0.25, offset=1.0, x_stride=stride)
        _, y = ol.rms_norm(f64(x)[:, :K], None, f64(w), 0.25, 1.0)
        check_rows(form, "bf16", y, NORM_DELTA, *got)


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("K,form", [(384, "f8_block"), (777, "f8_token"), (7168, "mx_f4"), (16512, "i8_token")])
def test_norm_sum_in_place(into, K, form):
    note(f"norm in place of {into} K={K} {form}")
    M = 6
    x, r, w = made(9, M, K, "bf16"), made(10, M, K, "bf16"), weight(11, K, "bf16")
    h, y = ol.rms_norm(f64(x), f64(r), f64(w), float(np.float32(1e-6)))
    target = x if into == "x" else r
    got = run_norm(form, "bf16", x, r, w, M, K, sum_out=target)
    check_rows(form, "bf16", y, NORM_DELTA, *got)
    assert (np.abs(f64(target) - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -23)).all()


@pytest.mark.parametrize("form", list(FORMS))
def test_norm_zeros_extremes_and_what_is_not_finite(form):
    """A row of zeros; one of tiny values; one of the type's largest; one with a NaN, one with an infinity,
    each beside ordinary rows that must not notice."""
    M, K = 6, 256
    note(f"norm special rows {form}")
    x = made(12, M, K, "fp16")
    x[1] = 0
    x[2] = 6e-8
    x[3] = 65504.0
    x[4, 17] = float("nan")
    x[5, 99] = float("inf")
    w = weight(13, K, "fp16")
    got = run_norm(form, "fp16", x, None, w, M, K)
    _, y = ol.rms_norm(f64(x), None, f64(w), float(np.float32(1e-6)))
    out, scale, nout, nscale = got
    head = lambda b, n: b[: n // M * 4] if b is not None else None  # noqa: E731
    each = lambda n: n // M * 4  # noqa: E731
    good = [head(out, nout), head(scale, nscale), each(nout), each(nscale)]
    check_rows(form, "fp16", y[:4], NORM_DELTA, *good)
    raw = out[:nout].view(M, -1)
    if form == "same":
        v = f64(raw.view(torch.float16).view(M, K))
        assert np.isnan(v[4]).all() and np.isnan(v[5, 99]) and (v[5, :99] == 0).all()
    elif form in ("f8_token", "f8_block"):
        v = f64(raw.view(torch.float8_e4m3fn).view(M, K))
        assert np.isnan(v[4]).all() and np.isnan(v[5, 99]) and (v[5, :99] == 0).all() and (v[5, 100:] == 0).all()
    elif form == "i8_token":
        assert (raw.view(torch.int8).view(M, K)[4:] == 0).all()
    else:
        e = scale[:nscale].view(M, -1)
        assert (e[4] == 255).all() and e[5, 3] == 255 and (e[5, :3] == 0).all()
        assert (raw[4] == 0).all() and ((raw[5] & (0x7F if form == "mx_f8" else 0x77)) == 0).all()  # (x / inf keeps the sign of x)


def test_norm_is_the_quantiser_after_the_norm():
    """Codes and scales of the fused call are those of the library's quantisers on its own fp32 values, where
    these are exact: ones times weights that are powers of two."""
    M, K = 4, 512
    note("norm of ones against the quantisers")
    x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.exp2(torch.randint(-6, 6, (K,), generator=torch.Generator().manual_seed(1)).float()).to(torch.bfloat16).cuda()
    y = (x.float() * w.float()).contiguous()
    for form, make in (("f8_token", lambda q, s: hq.hq_quantize_act(hq.HQ_DT_FP8_E4M3, M, K, y, q, s)),
                       ("f8_block", lambda q, s: hq.hq_quantize_act_blocks(hq.HQ_DT_FP8_E4M3, M, K, 128, y, q, s)),
                       ("mx_f8", lambda q, s: hq.hq_quantize_act_mx(hq.HQ_DT_FP8_E4M3, M, K, y, q, s)),
                       ("mx_f4", lambda q, s: hq.hq_quantize_act_mx(hq.HQ_DT_FP4_E2M1, M, K, y, q, s))):
        out, scale, nout, nscale = run_norm(form, "bf16", x, None, w, M, K, eps=0.0)
        q, s, _, _ = outputs(form, "bf16", M, K)
        make(q, s)
        torch.cuda.synchronize()
        assert torch.equal(out, q) and torch.equal(scale, s), form


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,I", [(1, 8), (3, 128), (5, 504), (4, 640), (2, 2048), (3, 2816), (2, 8192), (1, 9216), (1, 18432), (1, 65536)])
@pytest.mark.parametrize("form", [f for f in FORMS if f != "same"])
def test_swiglu_forms(form, rows, I, dtype):
    if I % (FORMS[form][2] or 1):
        pytest.skip("block scales need whole blocks")
    note(f"swiglu {form} {dtype} rows={rows} I={I}")
    x = made(14, rows, 2 * I, dtype, std=2.0).clamp(-30000, 30000)
    x[0, :4] = torch.tensor([-100.0, -60.0, 90.0, -0.0])
    odt, kind, _, _ = FORMS[form]
    out, scale, nout, nscale = outputs(form, dtype, rows, I)
    hq.hq_silu_mul_quant(DT[dtype][0], odt, kind, rows, I, x, out, scale)
    check_rows(form, dtype, ol.silu_mul(f64(x)), SILU_DELTA, out, scale, nout, nscale)


def test_norm_on_another_stream_and_in_a_graph():
    """Captured on a side stream and replayed with new inputs between eager calls: each replay as the eager call."""
    M, K = 9, 7168
    note("norm captured")
    x, r, w = made(15, M, K, "bf16"), made(16, M, K, "bf16"), weight(17, K, "bf16")
    desc = hq.norm_desc(hq.HQ_DT_BF16, hq.HQ_DT_FP8_E4M3, hq.HQ_ASCALE_PER_BLOCK128_F32)
    total = torch.empty_like(x)

    def call(o, s):
        hq.hq_rmsnorm(desc, M, K, x, K, w, o, s, residual=r, residual_stride=K, sum_out=total, sum_stride=K)

    out, scale, _, _ = outputs("f8_block", "bf16", M, K)
    want, want_s, _, _ = outputs("f8_block", "bf16", M, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, scale)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(out, scale)
    for i in range(3):
        x.copy_(made(20 + i, M, K, "bf16"))
        out.fill_(0x5A)
        scale.fill_(0x5A)
        g.replay()
        call(want, want_s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(scale, want_s)
