"""The cache calls refuse each single tensor that lies in host memory among device ones, before anything is queued, and take pinned ones."""
import numpy as np
import pytest
import torch

from cache_common import Cache, normal
from gpu_common import dev, require_gpu, say

pytestmark = pytest.mark.gpu


def test_single_host_tensors_are_refused():
    api = require_gpu()
    say("cache calls: host tensors")
    c = Cache("e4m3", "heads", 5, 16, 2, 64, 1)
    freq = dev(np.array(api.mxrope_freqs_host(64, 1e4)[0]))
    rope = api.Rope(64, freq)
    x = {"k": normal((3, 2, 64), "f16", 1), "v": normal((3, 2, 64), "f16", 2), "q": normal((3, 8, 64), "f16", 3), "q_out": normal((3, 8, 64), "f16", 4),
         "positions": dev(np.array([0, 5, 9], np.int32)), "seq": dev(np.arange(3, dtype=np.int32)), "table": dev(np.array([[0], [1], [2]], np.int32)),
         "lengths": dev(np.array([1, 6, 10], np.int32)), "starts": dev(np.zeros(3, np.int32)), "lse": torch.zeros(3, 8, device="cuda"),
         "workspace": torch.zeros(64, dtype=torch.uint8, device="cuda"), "pairs": dev(np.array([[3, 4]], np.int32))}

    def turn(z, rope=rope):
        api.mxrope_run(api.MX_F16, rope, z["q"], z["q_out"], z["positions"])

    def append(z, cache=c.c, rope=rope):
        api.mxkv_append_run(cache, api.MX_F16, z["k"], z["v"], z["positions"], z["table"], seq=z["seq"], rope=rope, q=z["q"], q_out=z["q_out"])

    def attend(z, cache=c.c):
        api.mxattn_decode_run(cache, api.MX_F16, z["q"], z["q_out"], z["table"], z["lengths"], 16, 0.1, lse=z["lse"], starts=z["starts"], workspace=z["workspace"])

    def copy(z, cache=c.c):
        api.mxkv_copy_run([cache], z["pairs"])

    for call, names in ((turn, "q q_out positions"), (append, "k v q q_out positions seq table"), (attend, "q q_out table lengths lse starts workspace"), (copy, "pairs")):
        call(x)
        for name in names.split():
            with pytest.raises(TypeError, match="GPU"):
                call(dict(x, **{name: x[name].cpu()}))
    for i in range(4):
        planes = list(c.planes + c.scales)
        planes[i] = planes[i].cpu()
        bad = api.KVCache(api.MX_E4M3, *planes)
        for call in (append, attend, copy):
            with pytest.raises(TypeError, match="GPU"):
                call(x, bad)
    for call in (turn, append):
        with pytest.raises(TypeError, match="GPU"):
            call(x, rope=api.Rope(64, freq.cpu()))
    attend(x)
    want = x["q_out"].clone()
    attend(dict(x, lengths=x["lengths"].cpu().pin_memory(), table=x["table"].cpu().pin_memory()))   # the GPU reads these
    assert torch.equal(x["q_out"], want)
