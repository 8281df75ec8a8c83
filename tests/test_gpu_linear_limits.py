"""GPU tests of the linear operators at the limits that they claim: 2^20 rows,
widths of 32768, 1024 groups, and tensors of more than 2^32 elements or bytes.
Exact, as in test_gpu_linear_shapes.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_sigmoid_amd as mx
from oracle import linear as ol
from tests.test_gpu_linear_shapes import check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


ROWS = 1 << 20
LIMITS = [
    ("fp8", ROWS, 3, 72, 80), ("fwd", ROWS, 3, 72, 80), ("dx", ROWS, 3, 72, 80), ("dw", ROWS, 3, 72, 80),
    # groups: through tiles, most of them empty, and in the few-row kernel
    ("fp8", 20000, 1024, 70, 144), ("fwd", 20000, 1024, 70, 72), ("dx", 20000, 1024, 72, 80), ("dw", 20000, 1024, 72, 80),
    ("fp8", 300, 1024, 200, 272), ("fwd", 300, 1024, 200, 136), ("dx", 300, 1024, 200, 136), ("dw", 300, 1024, 200, 136),
    ("fp8", 16, 1024, 24, 272), ("fwd", 16, 1024, 24, 136),
    # widths
    ("fp8", 40, 1, 32768, 32768), ("fwd", 40, 1, 32768, 32768), ("dx", 40, 1, 32768, 32768), ("dw", 40, 1, 32768, 32768),
    # weights past 2^32 bytes
    ("fp8", 900, 70, 8190, 8208), ("fwd", 900, 44, 8190, 8200), ("dx", 900, 44, 8184, 8200), ("dw", 900, 20, 8184, 8200),
    # rows past 2^32 bytes, of inputs and of outputs
    ("fp8", ROWS, 7, 40, 4112), ("fwd", 600000, 7, 40, 4104), ("dx", 600000, 7, 4104, 40), ("dx", 600000, 7, 40, 4104),
    ("dw", 600000, 7, 40, 4104), ("fwd", 600000, 7, 4104, 40),
]


@pytest.mark.parametrize("kind,rows,groups,N,K", LIMITS)
def test_products_at_the_limits(kind, rows, groups, N, K):
    print(f"[case] {kind} rows={rows} groups={groups} N={N} K={K}", flush=True)
    check(kind, rows, groups, N, K)


def _some(rows):
    return sorted({0, 1, 2, rows // 3, rows // 2, rows - 65, *range(rows - 5, rows)})


def _same(x, q, s, pick):
    """The picked rows of q and s are the correctly rounded codes and scales of x's."""
    xf = x[pick].float().cpu().numpy()
    rs = ol.quant_scales(xf)
    inv = np.float32(1) / ol.spread(rs, xf.shape[1], 1)
    codes = torch.from_numpy(xf * inv).to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(s[pick].cpu().numpy(), rs)
    assert torch.equal(q[pick].cpu(), codes)


@pytest.mark.parametrize("rows,K,ldx", [(ROWS, 4112, 4112), (ROWS, 128, 8192), (40000, 32768, 32768)])
def test_quant_past_32_bits(rows, K, ldx):
    """More than 2^32 bytes of codes, and of elements between the first and the last row."""
    print(f"[case] quant rows={rows} K={K} ldx={ldx}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    base = torch.empty(rows, ldx, dtype=torch.bfloat16, device="cuda")
    x = base[:, :K]
    x.copy_(torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8))
    q = torch.full((rows, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, ol.blocks(K)), -1.0, device="cuda")
    mx.moe_fp8_quant(x, q, s)
    torch.cuda.synchronize()
    _same(x, q, s, _some(rows))


def test_swiglu_quant_past_32_bits():
    """Gates of 100 pass their up value through: the codes are those of 100 * up."""
    rows, K = ROWS, 2064
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.full((rows, 2 * K), 100.0, dtype=torch.bfloat16, device="cuda")
    x[:, K:] = torch.randint(-128, 128, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    q = torch.full((rows, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, ol.blocks(K)), -1.0, device="cuda")
    mx.moe_fp8_swiglu_quant(x, q, s)
    torch.cuda.synchronize()
    pick = _some(rows)
    _same((100.0 * x[pick, K:].float()), q[pick], s[pick], list(range(len(pick))))
