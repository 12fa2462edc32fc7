"""Cosines and sines of the rotation keep fp32's relative precision, also where they are small."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from gpu_common import dev, require_gpu, say
from cache_common import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("inverse", [False, True])
def test_small_cosines_and_sines(layout, inverse):
    """x = (1, 0) turns into (cos w, sin w). Their error: the function's (2 ulp: 4 half steps), its correction's rounding (1) and, through
    the pair's exact products with 1 and 0, no more; with a half step to spare for each of the two stored values. The angle's
    own, in 64 bits: two roundings of w, and 2^-53 of a turn."""
    api = require_gpu()
    rot, tokens = 64, 4096
    freq = np.array(api.mxrope_freqs_host(rot, 10000.0)[0])
    r = api.Rope(rot, dev(freq), api.MXROPE_HALF if layout == "half" else api.MXROPE_PAIRS)
    pos = np.arange(tokens, dtype=np.int32)
    x = torch.zeros(tokens, 1, rot, device="cuda")
    first = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    x[:, 0, first] = 1.0
    out = torch.empty_like(x)
    say(f"rotary {layout}, inverse={inverse}: cosines and sines of {tokens} positions")
    api.mxrope_run(api.MX_F32, r, x, out, dev(pos), inverse=inverse)
    w = np.multiply.outer(pos.astype(np.longdouble), freq.astype(np.longdouble)) * (-1 if inverse else 1)
    worst = 0.0
    for at, f in ((first, np.cos), (second, np.sin)):
        want = f(w)
        bound = 6 * ref.U32 * np.abs(want) + 2.0 ** -52 * (np.abs(w) + 2 * np.pi)
        worst = max(worst, float((np.abs(f64(out)[:, 0, at] - want) / bound).max()))
    say(f"worst error / bound {worst:.3f}")
    assert worst <= 1.0
