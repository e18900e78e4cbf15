"""Whether a call with sinks cuts its units: no further than the table's own tokens ask for."""
import pytest

from gpu_util import require_gpu
from test_paged_sinks_gpu import Sinks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [1, 100, 5000])
@pytest.mark.parametrize("B,lens,new,Hq,H,D,cache", [(4, 600, 3, 8, 2, 128, None), (40, 1400, 8, 16, 4, 64, None),
                                                     (3, 900, 50, 8, 8, 64, "float8_e4m3fn")])
def test_sinks_past_the_table_are_the_whole_context(B, lens, new, Hq, H, D, cache, window):
    """The same bits as without a window; and, as there, no unit is cut: cut ones leave their
    parts (or that there are none) in the workspace for the join."""
    torch = require_gpu()
    from verify_dspark_markov_step_gb300 import _lib
    a = Sinks(torch, [lens - b for b in range(B)], [new] * B, Hq, H, D, 16, "bfloat16", cache, sinks=0)
    ws = _lib.workspace(_lib.paged_attention_workspace_bytes(B, Hq, H, D))
    made = []
    for sinks, w in ((0, 0), (a.dev[0].shape[1] * 16, window), (10 ** 6, window), (2 ** 31 - 1, window)):
        a.sinks = sinks
        ws.fill_(0x5A)
        a.out.fill_(3), a.lse.fill_(3)
        a.call(True, w, ws=ws)
        torch.cuda.synchronize()
        assert a.status.item() == 0
        made.append((a.out.clone(), a.lse.clone(), bool((ws == 0x5A).all())))
    assert made[0][2]  # (the table is short: nothing is cut)
    for out, lse, untouched in made[1:]:
        assert untouched
        assert torch.equal(out, made[0][0]) and torch.equal(lse, made[0][1])
