"""The 4-bit paged cache at the edges of what its calls allow."""
import math

import pytest
import torch

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests import kv4_format as F
from tests.test_gpu_kv4 import BF, F32, fill, gen, make, ok, randn, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", ["negative", "zero", "heads alike", "tokens alike"])
def test_prompts_that_the_tensor_copies_cannot_take(case):
    """Long bf16 segments whose scale or strides window attention's tensor-core form does not take stay where they are
    quick: nothing is read back, and the answers are those of the formula."""
    from tests.test_gpu_kv4_prompts import check, held
    g, n, T, hq, hk, d = gen(17), 300, 6000, 8, 2, 64
    cache, table = make([T], 64, hk, d)
    fill(cache, table, [T], BF, g)
    q = randn((n, hq, d), BF, g)
    scale = {"negative": -0.125, "zero": 0.0}.get(case, 0.125)
    if case == "heads alike":
        q = q[:, :1].expand(n, hq, d)
    if case == "tokens alike":
        q = q[:1].expand(n, hq, d)
    assert cache.workspace(q, table, [n], [T], scale=scale) < T * hk * d * 4
    out, lse = torch.empty((n, hq, d), dtype=BF, device="cuda"), torch.empty((n, hq), device="cuda")
    cache.attend(q, table, [n], [T], scale=scale, out=out, lse=lse)
    check(q, *held(cache, table, [T]), [n], [T], scale, out, lse)
    ok()
