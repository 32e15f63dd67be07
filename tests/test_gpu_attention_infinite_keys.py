"""A key that holds an infinity and so has no weight: scores of minus infinity, with head widths that fill a tile's rows and
widths that do not."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
from encoder_reference import attention, close
from test_gpu_attention import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hk,lens", [(2, 1, [90, 20, 200]), (1, 1, [20] * 30)])
@pytest.mark.parametrize("d", [8, 24, 32, 40, 104, 128])
def test_keys_at_minus_infinity_have_no_weight(d, hq, hk, lens, dtype):
    """As far below the others as a finite key can be, they give the same: weight 0 (float64: e^-745)."""
    print(f"[gpu] infinite keys d={d} hq={hq} {dtype}", flush=True)
    g = torch.Generator().manual_seed(d)
    n, dt = sum(lens), DT[dtype]
    q, k, v, dout = (torch.randn(n, h, d, generator=g).to(dt) for h in (hq, hk, hk, hq))
    q[..., -1] = 1.0 + q[..., -1].abs()
    offs = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    low = k.clone()
    low[5::7, :, -1] = -1e5
    k[5::7, :, -1] = float("-inf")
    op = rece.SequenceAttention(n, len(lens), hq, d, kv_heads=hk, dtype=dtype)
    args = [t.cuda() for t in (q, k, v, offs)]
    out, ws = op.forward(*args)
    _, dk, dv, _ = op.backward(*args, out, ws, dout.cuda())    # (dq: 0 times infinity)
    # a sequence's first row has nothing left where its own key is one of them: 0, and no gradient
    none = [a for a in offs[:-1].tolist() if a % 7 == 5]
    dout[none] = 0.0
    want = attention(q, low, v, offs.tolist(), op.scale, dout=dout)
    want["out"][0][none] = 0.0
    for name, t in (("out", out), ("dk", dk), ("dv", dv)):
        assert torch.isfinite(t).all(), name
        assert close(t, want[name]) <= 1.0, name
