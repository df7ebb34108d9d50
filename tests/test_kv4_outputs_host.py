"""Outputs of the 4-bit cache's calls that lie on what a call reads, or on each other, are refused (no GPU)."""
import pytest

from heterogeneous_compressed_kv_gb300 import kvpool as K
from tests.test_kv4_host import FAR, P16, attend, evict, heads

TABLE = FAR + (1 << 24)  # 3 rows of 4 ids, 4 apart
Q, OUT = P16, P16 + (1 << 22)  # 3 rows of 4 heads of 64 in 16 bits
AWAY = FAR * 8


@pytest.mark.parametrize("w", [FAR, FAR + 4096, TABLE, TABLE + 44, TABLE - 4 * 200 - 4 * 1024 + 4, Q, Q + 3 * 512 - 4, OUT + 512, OUT - 4, AWAY + 4])
def test_weights_of_attention_lie_apart(w):
    assert attend(w=w, lse=AWAY, work_too=False) == K.ERR_INVALID_ARG


@pytest.mark.parametrize("lse", [FAR, TABLE + 44, Q, Q - 44, Q + 3 * 512 - 4, OUT, OUT + 3 * 512 - 4, AWAY + 4 * 199, AWAY + 4 * 1024])
def test_log_sums_of_attention_lie_apart(lse):
    assert attend(w=AWAY, lse=lse, work_too=False) == K.ERR_INVALID_ARG


INDEX, OTABLE, OW, W = FAR * 5, FAR * 4, FAR * 3, P16  # where evict's arguments lie unless a test moves them


@pytest.mark.parametrize("kw", [dict(ow=FAR + 4096), dict(ow=TABLE + 44), dict(ow=OTABLE + 28), dict(ow=OTABLE - 4 * 1024),
                                dict(ow=INDEX), dict(ow=INDEX + 4 * 199), dict(ow=INDEX - 4 * 59), dict(index=OTABLE + 28), dict(index=OTABLE - 4 * 199),
                                dict(index=TABLE), dict(index=W), dict(index=W + 4 * 1024), dict(index=W - 4 * 199),
                                dict(index=W + 4 * (4096 + 1024 + 199)), dict(index=OW + 4 * 59), dict(index=OW + 4 * (4096 + 1024 + 59))])
def test_outputs_of_eviction_lie_apart(kw):
    """Two segments of up to 200 weights x 2 heads, 50 of which stay: index [2][2][50], weights behind up to 60."""
    kw = {x: y - y % 4 for x, y in kw.items()}
    assert evict(**kw) == K.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(index=W + 4 * 200), dict(index=W + 4 * 4096 + 4 * 200), dict(index=OW + 4 * 60), dict(ow=OTABLE + 32),
                                dict(ow=TABLE - 4 * 60),  # (its first 60 places end where the table starts)
                                dict(ow=INDEX + 4 * 200), dict(index=OTABLE + 32)])
def test_places_between_them_are_fine(kw):
    """An output may lie between the rows of another argument: such a call is not refused (and has no GPU to run on here)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert evict(**kw) == K.ERR_CUDA
