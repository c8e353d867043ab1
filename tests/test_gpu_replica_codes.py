"""8-bit codes and scales of the replica's RMS norm, bit for bit: what the
header says of them computed in binary32 on the host from the sum, the inverse
root and the scales that the call wrote, where a division is rounded once.
Helpers as in test_gpu_replica_ops.py."""
import pytest

from test_gpu_replica_ops import FLOATS, torch, v  # noqa: F401

pytestmark = pytest.mark.gpu

CODES = {"int8": 127.0, "e4m3": 448.0}


def _scales(torch, most, quant):  # noqa: F811
    """The largest |y| times the largest code's reciprocal, either rounded once."""
    return (most * (torch.ones_like(most) / torch.full_like(most, CODES[quant]))).clamp(min=2.0 ** -126)


def _call(torch, v, x, gamma, rows, cols, dtype, quant, group):  # noqa: F811
    groups = -(-cols // group) if group else 1
    r, s = torch.randn_like(x), torch.empty_like(x)
    codes = torch.empty(rows, cols, device="cuda", dtype=torch.int8 if quant == "int8" else torch.float8_e4m3fn)
    scales, rstd = torch.empty(rows, groups, device="cuda"), torch.empty(rows, device="cuda")
    v.vrcclRmsNormForward(x, r, gamma, s, None, rstd, rows, cols, dtype, "bfloat16", codes=codes, scales=scales, quant=quant, group=group)
    y = s.cpu().float() * rstd.cpu()[:, None] * gamma.cpu().float()  # (in the order of the kernel's products, each rounded)
    return y, codes.cpu(), scales.cpu()


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
@pytest.mark.parametrize("rows,cols,group", [(300, 128, 64), (900, 64, 0), (400, 5120, 128), (300, 4096, 0), (200, 4097, 32), (60, 1001, 0),
                                             (4, 40000, 64), (3, 40001, 0), (330, 9001, 128)])
def test_codes_bit_for_bit(torch, v, rows, cols, group, quant):  # noqa: F811
    """Of each walk over the rows: a code is y / scale rounded to binary32, then to the nearest code, even in the middle."""
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    for dtype in FLOATS:
        x = torch.randn(rows, cols, generator=gen, device="cuda").to(getattr(torch, dtype))
        # of few values, so that many quotients lie in the middle of two codes or next to it
        gamma = (1 + torch.randint(0, 8, (cols,), generator=gen, device="cuda") / 8).bfloat16()
        y, codes, scales = _call(torch, v, x, gamma, rows, cols, dtype, quant, group)
        at = y / scales.repeat_interleave(group or cols, 1)[:, :cols]
        if quant == "int8":
            assert torch.equal(codes.float(), at.round()), dtype
        else:
            assert torch.equal(codes.float(), at.to(torch.float8_e4m3fn).float()), dtype
        if group:  # (a row's largest is found before the inverse root is known: a rounding more)
            wide = torch.nn.functional.pad(y.abs(), (0, scales.shape[1] * group - cols)).view(rows, -1, group)
            assert torch.equal(scales, _scales(torch, wide.amax(2), quant)), dtype


@pytest.mark.parametrize("quant", ["int8", "e4m3"])
def test_codes_of_far_scales(torch, v, quant):  # noqa: F811
    """Scales over binary32's range; zeros; a group with an infinity beside others."""
    rows, cols, group = 64, 512, 32
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp2(torch.arange(16, device="cuda").repeat_interleave(32) * -6.0)  # 2^-90 .. 1 beside one another
    x[5], x[6, 32:64] = 0, 0
    gamma = torch.ones(cols, device="cuda", dtype=torch.bfloat16)
    s, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    codes = torch.empty(rows, cols, device="cuda", dtype=torch.int8 if quant == "int8" else torch.float8_e4m3fn)
    scales = torch.empty(rows, cols // group, device="cuda")
    v.vrcclRmsNormForward(x, None, gamma, s, None, rstd, rows, cols, "float32", "bfloat16", codes=codes, scales=scales, quant=quant, group=group)
    y = x.cpu() * rstd.cpu()[:, None]
    most = y.view(rows, -1, group).abs().amax(2)
    want = _scales(torch, most, quant)
    assert torch.equal(scales.cpu(), want)
    at = y / want.repeat_interleave(group, 1)
    assert torch.equal(codes.cpu().float(), at.round() if quant == "int8" else at.to(torch.float8_e4m3fn).float())
    x[7, 40] = float("inf")
    v.vrcclRmsNormForward(x, None, gamma, s, None, rstd, rows, cols, "float32", "bfloat16", codes=codes, scales=scales, quant=quant, group=group)
    fine = torch.isfinite(scales)
    assert not fine[7, 1] and fine.sum() == fine.numel() - 1
    assert torch.equal(torch.where(fine, scales, 0.0)[torch.arange(rows) != 7].cpu(), want[torch.arange(rows) != 7])
