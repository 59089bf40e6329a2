"""A step call whose workspace is refused enqueues nothing, its prompt chunks neither."""
import pytest

import synth
from harness import DeviceStep
from test_gpu_fp4 import F4Step, d32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pools", ["bf16", "e2m1"])
@pytest.mark.parametrize("fault", ["misaligned", "short", "none"])
def test_a_refused_workspace_leaves_the_outputs_alone(pools, fault):
    import paged_kv_gqa_row_gb300 as lnk
    w = synth.custom(seed=5, hq=8, hkv=2, head_dim=128, dec_lengths=[100, 40], chunks=[(0, 30)])
    dev = DeviceStep(w) if pools == "bf16" else F4Step(w)
    dev.append()
    dev.out.fill_(0x1234)
    need = lnk.lnk_paged_workspace_size(dev.desc, w.B)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    start, size = {"misaligned": (ws.data_ptr() + 128, need), "short": (ws.data_ptr(), need - 1), "none": (None, need)}[fault]
    with pytest.raises(lnk.LnkError) as e:
        lnk.lnk_paged_step_attn(dev.desc, dev.q_out, d32(w.ch_rows), d32(w.ch_positions), d32(w.ch_segments), dev.dec_positions,
                                dev.table, dev.k_pool, dev.v_pool, dev.out, None, None, w.P, w.B, 0, start, size, dev.status)
    assert e.value.status == 5
    torch.cuda.synchronize()
    assert bool((dev.out == 0x1234).all())
