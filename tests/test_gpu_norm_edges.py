"""The norm and rotation at the edges of its range: fp8 rows of tiny values, and every kernel form with what it
specialises (CUDA, through the C ABI), against fp64.

Tolerances: those of test_gpu_norm_rope.py for rows of ordinary size.  The fp8 scale of a tiny row is an fp32 number
that may be subnormal, so it is within an ulp or two (2^-22 of itself) and half the smallest step (2^-150) of max |y| /
448; a code is held against y over the scale that was returned: half an e4m3 step, 2^-4 of the quotient or 2^-10, and
1e-5 of it for the quotient's own fp32 rounding.
"""

import numpy as np
import pytest
import torch

from oracle.attention import norm_rope
from test_gpu_norm_rope import L, check, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check_tiny(y, codes, scale, what):
    """y [T, h, d] fp64 rows, their codes and scales."""
    c, s = codes.double().cpu().numpy(), scale.double().cpu().numpy()[..., None]
    top = np.abs(y).max(axis=-1, keepdims=True)
    want = np.where(top > 0, np.maximum(top / 448.0, 2.0 ** -149), 1.0)
    assert np.all(np.abs(s - want) <= 2.0 ** -22 * want + 2.0 ** -150), f"{what}: scales"
    assert np.all(np.isfinite(c)), f"{what}: codes that are not finite"
    assert np.all(c[y == 0] == 0), f"{what}: zeros"
    quot = y / s
    assert np.all(np.abs(c - quot) <= np.maximum(2.0 ** -4 * np.abs(quot), 2.0 ** -10) + 1e-5 * np.abs(quot)), what


@pytest.mark.parametrize("d", [64, 128, 192, 256, 512, 576, 1024])
def test_fp8_rows_of_tiny_values(L, d):  # noqa: F811
    """Rows whose scale is near or below the smallest normal fp32 number, zeros and subnormals among their values."""
    g = torch.Generator().manual_seed(d)
    tops = [5.2e-36, 5.4e-36, 1.4e-36, 1.3e-36, 1e-36, 1e-37, 2e-38, 1e-38, 3e-39, 2.0 ** -130, 2.0 ** -132, 2.0 ** -133]
    x = torch.empty(len(tops), 3, d, dtype=torch.float64).uniform_(-1, 1, generator=g)
    x *= torch.tensor(tops, dtype=torch.float64)[:, None, None]
    x[:, :, ::3] = 0.0
    x[:, 1, 1] = torch.tensor(tops, dtype=torch.float64)
    x[:, 2] = 0.0                                         # a row of one value alone
    x[:, 2, d - 1] = -torch.tensor(tops, dtype=torch.float64)
    x = x.to(torch.bfloat16).cuda()
    y, sc, _, _ = L.ls_norm_rope(x, None, fp8=True)
    check_tiny(x.double().cpu().numpy(), y, sc, "q")
    cache = torch.full((20, d), 1.0, device="cuda").to(torch.float8_e4m3fn)
    ks = torch.full((20,), 7.0, device="cuda")
    slots = torch.arange(len(tops), device="cuda") + 3
    L.ls_norm_rope(None, x[:, 1:2].contiguous(), k_cache=cache, k_scale=ks, slots=slots)
    check_tiny(x[:, 1:2].double().cpu().numpy(), cache[3:3 + len(tops)][:, None], ks[3:3 + len(tops), None], "k")
    assert torch.all(ks[:3] == 7) and torch.all(cache[:3].float() == 1)


def test_fp8_rows_of_tiny_values_rotated_and_normed(L):  # noqa: F811
    """The same behind a rotation by a quarter turn, and behind a norm whose weights are tiny: down to rows whose scale
    would be below the smallest fp32 number."""
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 0, :4] = torch.tensor([1e-37, -3e-37, 2e-38, 0.0])
    x[0, 1, 5] = 1e-38
    f = torch.zeros(64, device="cuda")                    # angle 0: the rotation leaves the values
    y, sc, _, _ = L.ls_norm_rope(x, None, torch.zeros(1, dtype=torch.int64, device="cuda"), f, fp8=True)
    check_tiny(x.double().cpu().numpy(), y, sc, "rotated")
    ones = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    ones[0, 0, 64:] = 0.0
    for w in (1e-36, 1e-38, 1e-41, 1e-43, 3e-45):
        wt = torch.full((128,), w, device="cuda")
        y, sc, _, _ = L.ls_norm_rope(ones, None, q_norm="rms", q_weight=wt, eps=0.0, fp8=True)
        val = float(wt[0]) * 2.0 ** 0.5
        c, s = y.double().cpu()[0, 0], float(sc[0, 0])
        assert torch.isfinite(c).all() and torch.all(c[64:] == 0), w
        # y itself is rounded to a multiple of 2^-149, the scale too; a code is half an e4m3 step off at most
        assert abs(s - max(val / 448, 2.0 ** -149)) <= 2.0 ** -150 + 2.0 ** -149 / 448 + 1e-6 * s, w
        assert torch.all((c[:64] * s - val).abs() <= 2.0 ** -149 + 2.0 ** -4 * val + 2.0 ** -10 * s), w


SHAPES = [
    # d, norm_dim, rope, rope_off: one, two, three, four and nine pieces a lane, the rotated part in the first, a middle
    # and the last step, across two steps, and at odd offsets
    (256, 256, 64, 0), (256, 256, 64, 192), (256, 128, 256, 0), (256, 256, 64, 101),
    (512, 512, 64, 0), (512, 512, 64, 256), (512, 512, 64, 448), (512, 512, 64, 224), (512, 448, 64, 3),
    (320, 320, 64, 0), (320, 320, 64, 128), (320, 320, 64, 256), (264, 264, 8, 256),
    (192, 192, 64, 0), (192, 192, 64, 64), (192, 128, 64, 128), (192, 192, 64, 32), (136, 136, 32, 104),
    (576, 576, 64, 0), (576, 512, 64, 480), (1024, 1024, 64, 224), (1024, 1024, 256, 256), (1024, 1000, 64, 960),
    (128, 128, 128, 0), (120, 120, 48, 72), (64, 32, 16, 48),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_every_form(L, shape, interleaved, fp8):  # noqa: F811
    d, nd, rope, off = shape
    s = make(9, 5, 2, d, rope, nd, seed=d + off)
    out = L.ls_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_norm="rms", k_norm="layer", norm_dim=nd,
                         q_weight=s["qw"], k_weight=s["kw"], k_bias=s["kb"], eps=1e-5, rope_off=off,
                         interleaved=interleaved, fp8=fp8)
    c = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    for x, norm, w, b, y, sc, name in ((s["q"], "rms", s["qw"], None, out[0], out[1], "q"),
                                       (s["k"], "layer", s["kw"], s["kb"], out[2], out[3], "k")):
        check(y, sc, norm_rope(c(x), c(s["pos"]), c(s["inv_freq"]), norm, nd, c(w), c(b), 1e-5, off, interleaved), name)
