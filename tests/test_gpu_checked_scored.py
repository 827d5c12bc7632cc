"""The scored router, its balance loss and gradients, and the 8-bit checkpoints in the bounds-checked
build (libmoe_checked.so): a child process loads it (MOE_LIBRARY) and runs small cases of every
kernel against the oracle; no check may fire."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.path.join(ROOT, "mixture_experts_layer_60_b200", "libmoe_checked.so")

CHILD = r"""
import os, sys, torch
sys.path.insert(0, os.getcwd())
import mixture_experts_layer_60_b200 as moe
assert moe.LIB_PATH.endswith("libmoe_checked.so"), moe.LIB_PATH
from tests import test_gpu_scored as TS, test_gpu_checkpoint8 as TC, test_gpu_scored_layer as TL
bf, f32 = torch.bfloat16, torch.float32
G = dict(n_groups=8, topk_groups=3, group_top=2)
for score in (TS.SIG, TS.SOFT):
    TS.test_route_scored(bf, score, 1, 64, 1, 1, {})
    TS.test_route_scored(bf, score, 8, 2048, 64, 6, dict(renorm=False))
    TS.test_route_scored(bf, score, 257, 256, 96, 8, G)
    TS.test_route_scored(bf, score, 1037, 2048, 64, 6, {})
    TS.test_route_scored(bf, score, 1301, 320, 257, 9, {})
    TS.test_route_scored(f32, score, 257, 256, 96, 8, G)
    for T, N, K, off in TS.SEQS:
        TS.test_balance_loss(score, T, N, K, off)
    for dt in (bf, f32):
        TS.test_route_scored_backward(dt, score, True, 130, 320, 61, 6, [3, 3, 60, 125])
        TS.test_route_scored_backward(dt, score, False, 515, 64, 320, 4, [0, 100, 400])
TS.test_route_scored_equal_keys_across_warps(1500)
TC.test_save8_packs_the_preactivations([0, 1, 15, 63, 64, 65, 130, 257, 17], 256, 128)
TC.test_save8_packs_the_preactivations([700], 512, 384)
TC.test_backward8([31, 32, 33, 0, 0, 300, 16], 256, 512)
TC.test_backward8_many_small_groups()
TL.test_training_step_of_a_scored_layer(TL.VARIANTS[2])
TL.test_training_step_with_8_bit_checkpoints(dict(score="softmax", balance_alpha=0.01))
torch.cuda.synchronize()
st = moe.moe_device_status()
assert st == 0, f"device error word {st}"
print("checked build ok")
"""


def test_checked_build_runs_the_scored_router_and_checkpoints():
    assert os.path.exists(CHECKED), "build it with `python -m mixture_experts_layer_60_b200.build --check-bounds`"
    env = dict(os.environ, MOE_LIBRARY=CHECKED)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build ok" in r.stdout
